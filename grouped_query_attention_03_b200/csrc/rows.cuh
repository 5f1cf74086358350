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
// mix of values - and rows_finish_kernel merges the parts in order:
//   m = max m_i, l = sum 2^(m_i - m) l_i, o = sum 2^(m_i - m) acc_i / l.
// scored: the parts also leave every scaled score s in the workspace, and
// the same kernel adds sum_rho 2^(s - m_rho) / l_rho to the cell's weight.
// The scores cost 8 bytes per row and cell (written, read) where reading the
// keys again would cost 2 d: less up to r * t_new = 32 rows at d = 128.
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
  float *acc;               // [slot][group_rows][d]
  float *scores;            // [B * Hkv][R][Cp] (scored), else NULL
  float *weights;           // [B,Hkv,C] (scored), else NULL
  int B, Hq, Hkv, C, d, t, r, R, window, tree;
  int Cp;                   // row pitch of scores: C rounded up to whole tiles
  int group_rows;           // rows one CTA works on (a slot's rows)
  int MG;                   // groups of group_rows rows per lane
  int ctas, min_tiles;      // tensor-core split (ctas CTAs share all tiles)
  int ns;                   // CUDA-core split (ns parts per lane), else 0
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
// lanes (b, g, group) one after the other; CTA c takes tiles [c per, (c+1)
// per).  Every CTA computes the same split from the lengths.
struct Split {
  long long total, per;
};

// Warp-wide.  `cum` of batch row b: tiles of the rows before it.
__device__ __forceinline__ Split split_of(const Params &p, int lane) {
  long long tot = 0;
  for (int b = lane; b < p.B; b += 32) tot += tiles_of(p, p.seq_lens[b]);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
  Split s;
  s.total = tot * p.Hkv * p.MG;
  s.per = (s.total + p.ctas - 1) / p.ctas;
  if (s.per < p.min_tiles) s.per = p.min_tiles;
  return s;
}

__device__ __forceinline__ long long tiles_before(const Params &p, int b_end, int lane) {
  long long tot = 0;
  for (int b = lane; b < b_end; b += 32) tot += tiles_of(p, p.seq_lens[b]);
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
  return tot * p.Hkv * p.MG;
}

// The parts of one (b, vl) lane group: np parts in slots s0, s0 + 1, ...
struct Parts {
  long long s0;
  int np;
};

// vl = g * MG + group.
__device__ __forceinline__ Parts parts_of(const Params &p, const Split &s, long long cum, int b,
                                          int vl) {
  Parts r;
  const long long L = (long long)b * p.Hkv * p.MG + vl;
  if (p.ns > 0) {
    r.s0 = L * p.ns;
    r.np = p.ns;
    return r;
  }
  const int nt = tiles_of(p, p.seq_lens[b]);
  const long long first = cum + (long long)vl * nt;
  const long long c0 = first / s.per;
  r.s0 = L + c0;
  r.np = nt == 0 ? 0 : (int)((first + nt - 1) / s.per - c0) + 1;
  return r;
}

// ------------------------------------------------------- merge and weights
constexpr int kFinishThreads = 256;
constexpr int kFinishCells = 4 * kFinishThreads;  // cells per CTA (weights)

// Blocks [0, merge_blocks): 8 rows each of a lane group; the rest: cells of a
// lane's weights.
template <typename T>
__global__ void __launch_bounds__(kFinishThreads)
    rows_finish_kernel(const Params p, int merge_blocks, int row_blocks, int cell_blocks) {
  __shared__ Split s_split;
  __shared__ long long s_cum;
  __shared__ float s_m[kFinishThreads], s_inv[kFinishThreads];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int LPB = p.Hkv * p.MG;
  const bool merging = (int)blockIdx.x < merge_blocks;
  const long long i = merging ? blockIdx.x : blockIdx.x - merge_blocks;
  const long long lg = merging ? i / row_blocks : i / cell_blocks;  // lane group, or lane
  const int part = (int)(i - lg * (merging ? row_blocks : cell_blocks));
  const int b = (int)(lg / (merging ? LPB : p.Hkv));
  const int x = (int)(lg - (long long)b * (merging ? LPB : p.Hkv));  // vl, or g
  const int n = p.seq_lens[b];
  if (!length_ok(p, n)) return;  // its output is zeroed by the split kernel
  if (!merging && part * kFinishCells >= n) return;
  if (p.ns == 0 && warp == 0) {
    const Split s = split_of(p, lane);
    const long long cum = tiles_before(p, b, lane);
    if (lane == 0) {
      s_split = s;
      s_cum = cum;
    }
  }
  __syncthreads();

  if (merging) {
    const Parts pt = parts_of(p, s_split, s_cum, b, x);
    const int g = x / p.MG, grp = x - g * p.MG;
    const int row = part * (kFinishThreads / 32) + warp;  // in the group
    const int rho = grp * p.group_rows + row;
    if (pt.np <= 1 || row >= p.group_rows || rho >= p.R) return;
    float m = -INFINITY;
    for (int j = lane; j < pt.np; j += 32) m = fmaxf(m, p.ml[(pt.s0 + j) * p.group_rows + row].x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float l = 0.f, a[GQA_MAX_HEAD_DIM / 32];
#pragma unroll
    for (int c = 0; c < GQA_MAX_HEAD_DIM / 32; ++c) a[c] = 0.f;
    const float *acc = p.acc + (pt.s0 * p.group_rows + row) * p.d;
    const long long step = (long long)p.group_rows * p.d;
    for (int j0 = 0; j0 < pt.np; j0 += 32) {
      const int nj = min(32, pt.np - j0);
      float e = 0.f, lw = 0.f;
      if (lane < nj) {
        const float2 y = p.ml[(pt.s0 + j0 + lane) * p.group_rows + row];
        // a part without keys has l = 0; one whose scores are all NaN keeps it
        e = y.x == -INFINITY ? (y.y != 0.f ? 1.f : 0.f) : exp2f(y.x - m);
        lw = y.y;
      }
#pragma unroll 4
      for (int j = 0; j < nj; ++j) {
        const float ej = __shfl_sync(0xffffffffu, e, j), lj = __shfl_sync(0xffffffffu, lw, j);
        if (ej == 0.f) continue;  // an empty part: its acc is not written
        l = fmaf(ej, lj, l);
#pragma unroll
        for (int c = 0; c < GQA_MAX_HEAD_DIM / 32; ++c)
          if (c * 32 + lane < p.d) a[c] = fmaf(ej, acc[(j0 + j) * step + c * 32 + lane], a[c]);
      }
    }
    T *o = (T *)p.o + (((long long)b * p.Hq + (long long)g * p.r) * p.t + rho) * p.d;
    const float inv = 1.f / l;
    const bool dead = l == 0.f;  // no key at all: zero
#pragma unroll
    for (int c = 0; c < GQA_MAX_HEAD_DIM / 32; ++c)
      if (c * 32 + lane < p.d) o[c * 32 + lane] = from_f32<T>(dead ? 0.f : a[c] * inv);
    return;
  }

  // weights of cells [j, j + 4) of lane (b, g)
  const int g = x, j = part * kFinishCells + threadIdx.x * 4;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < p.R; r0 += kFinishThreads) {
    const int rho = r0 + threadIdx.x;
    __syncthreads();
    if (rho < p.R) {
      const int grp = rho / p.group_rows, row = rho - grp * p.group_rows;
      const Parts pt = parts_of(p, s_split, s_cum, b, g * p.MG + grp);
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < pt.np; ++k) m = fmaxf(m, p.ml[(pt.s0 + k) * p.group_rows + row].x);
      for (int k = 0; k < pt.np; ++k) {
        const float2 y = p.ml[(pt.s0 + k) * p.group_rows + row];
        l = fmaf(y.x == -INFINITY ? (y.y != 0.f ? 1.f : 0.f) : exp2f(y.x - m), y.y, l);
      }
      s_m[threadIdx.x] = m == -INFINITY ? 0.f : m;
      s_inv[threadIdx.x] = l == 0.f ? 0.f : 1.f / l;
    }
    __syncthreads();
    if (j >= n) continue;
    const int nr = min(kFinishThreads, p.R - r0);
    const float *s = p.scores + ((long long)(b * p.Hkv + g) * p.R + r0) * p.Cp + j;
#pragma unroll 4
    for (int k = 0; k < nr; ++k) {
      const float4 y = *reinterpret_cast<const float4 *>(s + (long long)k * p.Cp);
      const float m = s_m[k], inv = s_inv[k];
      w[0] = fmaf(exp2f(y.x - m), inv, w[0]);
      w[1] = fmaf(exp2f(y.y - m), inv, w[1]);
      w[2] = fmaf(exp2f(y.z - m), inv, w[2]);
      w[3] = fmaf(exp2f(y.w - m), inv, w[3]);
    }
  }
  float *out = p.weights + ((long long)b * p.Hkv + g) * p.C + j;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (j + k < n) out[k] += w[k];
}

}  // namespace rows
}  // namespace gqa
