// rows.cuh -- what the kernels behind gqa_decode_tree and gqa_decode_scored
// share: which keys a row may read, how the work is split, and the merge.
//
// A lane is one (b, g): the R = r * t_new rows of the KV group's r query
// heads, row rho = head * t_new + i, i the drafted node (tree) or the new
// row (scored); in q and o they are R consecutive rows.  The lane's keys are
// the cells [lo0, n_b) and then, for a tree, its t_new drafted rows.
//   tree    node i at depth m reads cells >= n_b + m - (w - 1) (window w) and
//           the drafts of its own line, the last w of it
//   scored  row i reads cells [0, n_b - t_new + i]
// The keys are split over CTAs, each writes (m, l, acc) of its part - the
// maximum of the scaled scores (log2 units), the sum of 2^(s - m), and the
// mix of values - to the workspace, and the parts are merged in order:
//   m = max m_i, l = sum 2^(m_i - m) l_i, o = sum 2^(m_i - m) acc_i / l.
// Few small parts: by the last CTA to count a lane's parts (the counters are
// zero between calls, the last count resets them).  Many or large ones: by
// rows_finish_kernel, all SMs together (p.finish).  Either way the bits do
// not depend on who merges, and no CTA waits for another.
// scored: every row's m and 1 / l are kept, and a second kernel adds
// sum_rho 2^(s - m_rho) / l_rho to each cell's weight: from the scores, left
// in the workspace by the parts (rows_weigh_kernel), or from the keys, read
// once more (rows_weigh_tc.cuh; rows_weigh_keys_kernel on CUDA cores).
#pragma once

#include "common.cuh"

namespace gqa {
namespace rows {

constexpr int kTile = 128;   // keys per tile of the tensor-core kernel
constexpr int kMaxNodes = GQA_MAX_TREE;

struct Params {
  const void *q, *k, *v;    // k, v: the cache [B,Hkv,C,d]
  const void *kd, *vd;      // drafts [B,Hkv,t,d] (tree)
  const int32_t *parents;   // [B,t] or NULL (tree)
  const int32_t *seq_lens;
  void *o;
  int32_t *status;
  float2 *ml;               // [slot][group_rows]
  float *acc;               // [slot][ceil(d / 4)][group_rows][4]
  int2 *groups;             // [B * Hkv * MG] (p.finish): the CTA of a lane group's
                            // first part and the number of its parts
  int *counters;            // [kCounters], zero at start and end: parts done
  float2 *lse;              // [B * Hkv][R] (scored): m and 1 / l of every row
  float *scores;            // [B * Hkv][R][Cp] (scored, few rows), else NULL
  float *weights;           // [B,Hkv,C] (scored), else NULL
  int B, Hq, Hkv, C, d, t, r, R, window, tree;
  int Cp;                   // row pitch of scores: C rounded up to whole tiles
  int group_rows;           // rows one CTA works on (a slot's rows)
  int MG;                   // groups of group_rows rows per lane
  int ctas, pad;            // tensor-core split (ctas CTAs share all tiles)
  int ns;                   // CUDA-core split (ns parts per lane), else 0
  int vec;                  // CUDA cores: rows are whole aligned 16-byte vectors
  int finish;               // rows_finish_kernel merges
  float scale_log2;
};

// Keys and tiles of a sequence of length n; 0 for one that is refused.
__device__ __forceinline__ bool length_ok(const Params &p, int n) {
  return n >= (p.tree ? 0 : p.t) && n <= p.C;
}
__device__ __forceinline__ int first_cell(const Params &p, int n) {
  return p.window > 0 ? max(0, n - (p.window - 1)) : 0;
}
__device__ __forceinline__ int tiles_of(const Params &p, int n) {
  if (!length_ok(p, n)) return 0;
  return (n - first_cell(p, n) + kTile - 1) / kTile + p.tree;
}

// A node's line in the tree: the drafts it may read, as bits, and its depth.
struct Line {
  uint32_t bits[kMaxNodes / 32];
  int depth;   // -1: padding, or refused
  bool refused;
};

// par: the sequence's parents (shared memory), or NULL for a chain.
__device__ __forceinline__ Line line_of(const int32_t *par, int i, int window) {
  Line ln;
#pragma unroll
  for (int w = 0; w < kMaxNodes / 32; ++w) ln.bits[w] = 0u;
  ln.depth = -1;
  ln.refused = false;
  int steps = 0;
  for (int at = i;; ++steps) {
    if (window < 0 || steps < window) {
#pragma unroll
      for (int w = 0; w < kMaxNodes / 32; ++w)
        if ((at >> 5) == w) ln.bits[w] |= 1u << (at & 31);
    }
    const int up = par ? par[at] : at - 1;
    if (up == -1) break;
    if (up < 0 || up >= at) {  // padding (of the node itself: no fault), or no parent
      ln.refused = !(up == -2 && at == i);
#pragma unroll
      for (int w = 0; w < kMaxNodes / 32; ++w) ln.bits[w] = 0u;
      return ln;
    }
    at = up;
  }
  ln.depth = steps;
  return ln;
}

// ------------------------------------------------- the tensor-core split
// The tiles of all lanes laid end to end, batch row by batch row, a row's
// lane groups (b, g, group) one after the other; CTA c takes the positions
// [c per, (c+1) per).  Every CTA computes the same split from the lengths.
//   running   each lane group is preceded by `pad` virtual tiles that carry no
//             work (what a lane group costs a CTA besides its tiles: queries,
//             masks, O's way out), and a CTA's range may hold the end of one
//             group and the start of another
//   aligned   each lane group starts at a CTA of its own (its extent is a
//             multiple of per): no CTA changes groups on the way, which costs
//             it about 4 us each time.  Taken for up to 32 sequences where a
//             CTA's share grows by at most a quarter (the fewer CTAs then
//             stream as fast as memory allows: 1.0 us a tile against the 1.4
//             that 148 CTAs share it at).
// a / b, both non-negative: the 64-bit divide is a long software sequence, and
// here nearly every pair fits 32 bits.
__device__ __forceinline__ long long udiv(long long a, long long b) {
  if (((unsigned long long)a | (unsigned long long)b) < (1ull << 32))
    return (long long)((unsigned)a / (unsigned)b);
  return a / b;
}

struct Split {
  long long total, per;
  int pad, aligned;
};

__device__ __forceinline__ long long extent_of(const Params &p, const Split &s, int n) {
  const int nt = tiles_of(p, n);
  if (nt == 0) return 0;
  return s.aligned ? udiv(nt + s.per - 1, s.per) * s.per : nt + s.pad;
}

// Warp-wide; the first kLenCache lengths are left in `cache` on the way.
constexpr int kLenCache = 128;
__device__ __forceinline__ Split split_of(const Params &p, int lane, int32_t *cache) {
  long long tot = 0;
  int nt = 0, filled = 0;
  for (int b = lane; b < p.B; b += 32) {
    const int n = __ldcg(p.seq_lens + b);
    if (b < kLenCache) cache[b] = n;
    nt = tiles_of(p, n);
    tot += nt;
    filled += nt > 0;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
  filled = __reduce_add_sync(0xffffffffu, filled);
  __syncwarp();
  const long long LPB = (long long)p.Hkv * p.MG;
  Split s;
  s.pad = p.pad;
  s.aligned = 0;
  s.total = (tot + (long long)filled * p.pad) * LPB;
  s.per = udiv(s.total + p.ctas - 1, p.ctas);
  if (s.per < 1) s.per = 1;
  if (p.B <= 32 && s.per > 1 && filled * LPB <= p.ctas && s.total < (1 << 24)) {
    // the smallest share with which whole CTAs suffice, if it is near
    const int most = (int)(s.per + s.per / 4);
    int per = max((int)udiv(tot * LPB + p.ctas - 1, p.ctas), 1), used = 0;
    for (int i = 0; i < 8 && per <= most; ++i) {
      used = (int)LPB * (int)__reduce_add_sync(0xffffffffu, (unsigned)((nt + per - 1) / per));
      if (used <= p.ctas) {
        // as small as gives every group the same number of parts
        const int np = max(1, (nt + per - 1) / per);
        per = max((int)__reduce_max_sync(0xffffffffu, (unsigned)((nt + np - 1) / np)), 1);
        s.aligned = 1;
        s.pad = 0;
        s.per = per;
        s.total = (long long)used * per;
        break;
      }
      per = max(per + 1, per * used / p.ctas);
    }
  }
  return s;
}

// ----------------------------------------------------------------- counting
// One counter per lane group in several parts: indexed by the CTA of its
// first part (tensor cores: a CTA starts at most one such group) or by the
// group itself (CUDA cores: cut only while there are at most kCounters / 2).
constexpr int kCounters = 1024;

__device__ __forceinline__ void fence_acq_rel_gpu() {
  asm volatile("fence.acq_rel.gpu;" ::: "memory");
}

// By one thread, after a barrier behind the stores of the part: true if this
// was the last of np, whose loads then see every part (after a barrier).
__device__ __forceinline__ bool count_part(int *counter, int np) {
  fence_acq_rel_gpu();
  const bool last = atomicAdd(counter, 1) == np - 1;
  if (last) {
    *counter = 0;
    fence_acq_rel_gpu();
  }
  return last;
}

// A part's weight 2^(m_i - m).  One without keys has l = 0; one whose scores
// are all NaN has no maximum either, and keeps its sum.
__device__ __forceinline__ float part_weight(float2 ml, float m) {
  return ml.x == -INFINITY ? (ml.y != 0.f ? 1.f : 0.f) : exp2f(ml.x - m);
}

// Columns [4 c0, ...) of a row over np parts: U groups of 4 columns, wpc
// apart, J parts in flight.
template <int U, int J>
__device__ __forceinline__ void merge_columns(const Params &p, const float2 *ml, const float4 *acc,
                                              int np, int d4, int wpc, int c0, float m, float *row,
                                              float *l_out) {
  float a[U][4], l = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) a[u][0] = a[u][1] = a[u][2] = a[u][3] = 0.f;
  for (int j0 = 0; j0 < np; j0 += J) {
    float2 y[J];
    float4 v[J][U];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      y[j] = make_float2(-INFINITY, 0.f);
      if (j0 + j < np) y[j] = __ldcg(&ml[(long long)(j0 + j) * p.group_rows]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (j0 + j < np && c0 + u * wpc < d4)
          v[j][u] = __ldcg(&acc[((long long)(j0 + j) * d4 + c0 + u * wpc) * p.group_rows]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (j0 + j >= np) break;
      const float e = part_weight(y[j], m);
      l = fmaf(e, y[j].y, l);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + u * wpc < d4) {
          a[u][0] = fmaf(e, v[j][u].x, a[u][0]);
          a[u][1] = fmaf(e, v[j][u].y, a[u][1]);
          a[u][2] = fmaf(e, v[j][u].z, a[u][2]);
          a[u][3] = fmaf(e, v[j][u].w, a[u][3]);
        }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: no key at all
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + u * wpc < d4)
      *reinterpret_cast<float4 *>(row + (c0 + u * wpc) * 4) =
          make_float4(a[u][0] * inv, a[u][1] * inv, a[u][2] * inv, a[u][3] * inv);
  *l_out = l;
}

// Merges np parts (slots s0 ..) of a lane group's nrows (<= 32 NW) rows: into
// tile[row * pitch + column] in shared memory, and lse.  NW warps; each takes
// 32 rows and every wpc-th group of 4 columns, a lane per row, so loads are
// 512 consecutive bytes.  What it takes is round trips to L2 (the parts are
// other SMs' last stores), so 16 loads are in flight at a time, over columns
// or over parts.
template <int NW>
__device__ __forceinline__ void merge_parts(const Params &p, long long s0, int np, int nrows,
                                            int warp, float *tile, int pitch, float2 *lse) {
  const int lane = threadIdx.x & 31;
  const int chunks = (nrows + 31) / 32, wpc = NW / chunks;  // warps per 32 rows
  const int chunk = warp / wpc, sub = warp - chunk * wpc;
  const int row = chunk * 32 + lane, d4 = (p.d + 3) / 4;
  if (chunk >= chunks || row >= nrows) return;
  const float2 *ml = p.ml + s0 * p.group_rows + row;
  float m = -INFINITY, l = 0.f;
#pragma unroll 8
  for (int j = 0; j < np; ++j) m = fmaxf(m, __ldcg(&ml[(long long)j * p.group_rows].x));
  const float4 *acc = reinterpret_cast<const float4 *>(p.acc) + s0 * d4 * p.group_rows + row;
  if (np <= 4) {
    for (int c0 = sub; c0 < d4; c0 += 4 * wpc)
      merge_columns<4, 4>(p, ml, acc, np, d4, wpc, c0, m, tile + row * pitch, &l);
  } else {
    for (int c0 = sub; c0 < d4; c0 += 2 * wpc)
      merge_columns<2, 8>(p, ml, acc, np, d4, wpc, c0, m, tile + row * pitch, &l);
  }
  if (lse && sub == 0) lse[row] = make_float2(m == -INFINITY ? 0.f : m, l == 0.f ? 0.f : 1.f / l);
}

// ------------------------------------------------------------------- finish
// Block (lane group, 32 rows, 8 / WP groups of 4 columns): WP warps share a group
// of columns, each with every WP-th part, a lane per row.  Up to 16 parts are
// fetched at once, their statistics and sums together, so that the kernel is
// two round trips to L2 (which group, its parts); more parts per warp take a
// pass over the statistics first.
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kFinishRows = 32;

template <typename T, int WP>
__global__ void __launch_bounds__(kFinishThreads)
    rows_finish_kernel(const Params p, int row_blocks, int col_blocks) {
  constexpr int WC = kFinishWarps / WP, COLS = 4 * WC;
  __shared__ __align__(16) float tile[kFinishRows][COLS + 4];
  __shared__ float4 s_acc[kFinishWarps][kFinishRows];
  __shared__ float2 s_ml[kFinishWarps][kFinishRows];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wc = warp / WP, wp = warp % WP;
  int i = blockIdx.x;
  const int cb = i % col_blocks;
  i /= col_blocks;
  const int rb = i % row_blocks, L = i / row_blocks;
  const int2 x = p.groups[L];
  const int ln = L / p.MG, grp = L - ln * p.MG, np = x.y;
  // (A refused sequence's entry is not written; every other one is, also after
  // a wait that ran out, since the writing warp walks on.)
  if (!length_ok(p, p.seq_lens[ln / p.Hkv])) return;
  if (np < 2) return;
  const int rho0 = grp * p.group_rows + rb * kFinishRows;  // first row of the lane
  const int nrows = min(min(kFinishRows, p.group_rows - rb * kFinishRows), p.R - rho0);
  if (nrows <= 0) return;
  const int d4 = p.d / 4, c4 = cb * WC + wc;  // d is 64 or 128
  float m = -INFINITY, l = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane < nrows) {
    const long long s0 = (long long)L + x.x;  // the first part's slot
    const int row = rb * kFinishRows + lane;
    const float2 *ml = p.ml + s0 * p.group_rows + row;
    const float4 *acc =
        reinterpret_cast<const float4 *>(p.acc) + (s0 * d4 + c4) * p.group_rows + row;
    constexpr int J = 16;
    const long long step = (long long)d4 * p.group_rows;
    float2 y[J];
    float4 v[J];
    auto fetch = [&](int j0) {  // parts j0, j0 + WP, ...
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (j0 + j * WP < np) {
          y[j] = ml[(long long)(j0 + j * WP) * p.group_rows];
          v[j] = acc[(j0 + j * WP) * step];
        } else {
          y[j] = make_float2(-INFINITY, 0.f);
          v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    fetch(wp);
#pragma unroll
    for (int j = 0; j < J; ++j) m = fmaxf(m, y[j].x);
#pragma unroll 16
    for (int j = wp + J * WP; j < np; j += WP) m = fmaxf(m, ml[(long long)j * p.group_rows].x);
    for (int j0 = wp; j0 < np; j0 += J * WP) {
      if (j0 > wp) fetch(j0);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j0 + j * WP >= np) break;
        const float e = part_weight(y[j], m);
        l = fmaf(e, y[j].y, l);
        a.x = fmaf(e, v[j].x, a.x);
        a.y = fmaf(e, v[j].y, a.y);
        a.z = fmaf(e, v[j].z, a.z);
        a.w = fmaf(e, v[j].w, a.w);
      }
    }
  }
  if constexpr (WP > 1) {  // the warps' sums, in order
    s_ml[warp][lane] = make_float2(m, l);
    s_acc[warp][lane] = a;
    __syncthreads();
    if (wp == 0) {
#pragma unroll
      for (int u = 1; u < WP; ++u) m = fmaxf(m, s_ml[warp + u][lane].x);
      l = 0.f;
      a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < WP; ++u) {
        const float2 y = s_ml[warp + u][lane];
        const float4 v = s_acc[warp + u][lane];
        const float e = part_weight(y, m);
        l = fmaf(e, y.y, l);
        a.x = fmaf(e, v.x, a.x);
        a.y = fmaf(e, v.y, a.y);
        a.z = fmaf(e, v.z, a.z);
        a.w = fmaf(e, v.w, a.w);
      }
    }
  }
  if (wp == 0 && lane < nrows) {
    const float inv = l == 0.f ? 0.f : 1.f / l;  // 0: no key at all
    *reinterpret_cast<float4 *>(&tile[lane][wc * 4]) =
        make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if (p.lse && c4 == 0)
      p.lse[(long long)ln * p.R + rho0 + lane] =
          make_float2(m == -INFINITY ? 0.f : m, l == 0.f ? 0.f : 1.f / l);
  }
  __syncthreads();
  T *o = (T *)p.o + ((long long)ln * p.R + rho0) * p.d + cb * COLS;
  for (int e = threadIdx.x; e < nrows * (COLS / 2); e += kFinishThreads) {
    const int k = e / (COLS / 2), col = 2 * (e % (COLS / 2));
    *reinterpret_cast<uint32_t *>(o + (long long)k * p.d + col) =
        pack_bf16(tile[k][col], tile[k][col + 1]);
  }
}

// ------------------------------------------------------------------ weights
constexpr int kWeighThreads = 256;
constexpr int kWeighCells = 4 * kWeighThreads;  // cells per CTA

__global__ void __launch_bounds__(kWeighThreads) rows_weigh_kernel(const Params p, int cell_blocks) {
  __shared__ float s_m[kWeighThreads], s_inv[kWeighThreads];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int ln = blockIdx.x / cell_blocks, part = blockIdx.x - ln * cell_blocks;  // lane (b, g)
  const int b = ln / p.Hkv;
  // cells [j, j + 4) of the lane: the first rows' scores and the weights are
  // on their way while the length and the rows' statistics are read
  constexpr int U = 8;
  const int j = part * kWeighCells + threadIdx.x * 4;
  const float *s0 = p.scores + (long long)ln * p.R * p.Cp + min(j, p.Cp - 4);
  float *out = p.weights + (long long)ln * p.C + j;
  float4 y[U];
  float old[4];
#pragma unroll
  for (int u = 0; u < U; ++u)
    y[u] = u < p.R ? *reinterpret_cast<const float4 *>(s0 + (long long)u * p.Cp)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 4; ++k) old[k] = j + k < p.C ? out[k] : 0.f;
  const int n = p.seq_lens[b];
  if (!length_ok(p, n) || part * kWeighCells >= n) return;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < p.R; r0 += kWeighThreads) {
    const int rho = r0 + threadIdx.x;
    __syncthreads();
    if (rho < p.R) {
      const float2 x = p.lse[(long long)ln * p.R + rho];
      s_m[threadIdx.x] = x.x;
      s_inv[threadIdx.x] = x.y;
    }
    __syncthreads();
    const int nr = min(kWeighThreads, p.R - r0);
    for (int k0 = 0; k0 < nr; k0 += U) {
      if (r0 + k0 > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k0 + u < nr) y[u] = *reinterpret_cast<const float4 *>(s0 + (long long)(r0 + k0 + u) * p.Cp);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + u >= nr) break;
        const float m = s_m[k0 + u], inv = s_inv[k0 + u];
        w[0] = fmaf(exp2f(y[u].x - m), inv, w[0]);
        w[1] = fmaf(exp2f(y[u].y - m), inv, w[1]);
        w[2] = fmaf(exp2f(y[u].z - m), inv, w[2]);
        w[3] = fmaf(exp2f(y[u].w - m), inv, w[3]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (j + k < n) out[k] = old[k] + w[k];
}

}  // namespace rows
}  // namespace gqa
