// rows_splitk.cuh -- tcgen05/TMEM split-K attention of up to 128 query rows
// per head over a cache: gqa_decode_tree and gqa_decode_scored for bf16 with
// d = 64 or 128 (sm_100a).  Which keys a row reads, the split over CTAs and
// the merge are in rows.cuh.
//
// The rows of a KV group (r heads x t_new rows, consecutive in q) fill the
// 128 TMEM lanes of one or two row tiles (NT), so every K and V tile is
// fetched once for all of them; more rows make more lane groups.  A CTA
// walks its range of 128-key tiles, one per SM:
//   warp 0      TMA producer: a segment's Q tiles, then K and V tiles into
//               STAGES-deep rings (128-byte swizzle, no multicast)
//   warp 1      one lane issues tcgen05.mma: S = Q K^T (M = N = 128, K = d)
//               into TMEM, and O += P V with P read from TMEM
//   warp 2      zeroes the outputs of refused sequences, reports them
//   4 NT warps  softmax, one thread per row: loads its S row, masks edge
//               tiles, rescales O when its maximum grew by more than 2^8,
//               writes bf16 P over S; at the end of a segment the O row goes
//               out (a lane group in one part) or to the workspace
// TMEM: NT = 1 has two S buffers, so S(j+1) is computed under the softmax of
// tile j; NT = 2 has one per row tile, and the two tiles take turns.
//
// Bound by HBM while a group has at most about 256 rows: a 128-key tile is
// 4 d * 128 bytes, 1.5 us of an SM's share of the bandwidth at d = 128,
// against 0.4 us of MMA and about 0.8 us of softmax per row tile.
//
// What a row may not read never reaches it: its scores are masked by a
// select, and since 0 * NaN is not 0, value rows of an edge tile that some
// row may not read are cleared in shared memory when they are not finite
// (or not anybody's) and added to the rows that may read them from global
// memory at the end of the segment (add_unfinite).
#pragma once

#include <cuda.h>

#include "rows.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace gqa {
namespace rows {

constexpr int kM = 128;                    // rows per row tile
constexpr uint32_t kTmemCols = 512;
constexpr float kLazyRescale = 8.0f;       // log2 units
// Registers per thread of the NT = 2 kernel after the split: 128 * low + 256 *
// high must not exceed its 384 threads times the 168 they are launched with.
constexpr int kRegsLow = 72, kRegsHigh = 216;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= 384 * 168, "register split");
constexpr int kUnfinite = 4;               // edge tiles of a segment at most

template <int D, int NT>
struct TcCfg {
  static constexpr int THREADS = 128 + 128 * NT;
  static constexpr int KB = D / 64;            // 64-column blocks
  static constexpr int BLK = 128 * 128;        // 128 rows x 128 B
  static constexpr int TILE = KB * BLK;        // a Q, K or V tile
  // as many stages of K and V as fit beside Q in 224 KB
  static constexpr int STAGES = (224 * 1024 - NT * TILE) / (2 * TILE) < 6
                                    ? (224 * 1024 - NT * TILE) / (2 * TILE) : 6;
  static constexpr int OFF_K = NT * TILE;
  static constexpr int OFF_V = OFF_K + STAGES * TILE;
  static constexpr int SMEM = OFF_V + STAGES * TILE + 1024;  // + alignment
  static constexpr uint32_t TM_O = 256;
  static_assert(TM_O + NT * D <= kTmemCols, "S and O must fit in TMEM");
};

struct Unfinite {  // value rows of one edge tile cleared for the MMA
  int tile;
  uint32_t bits[4];
};

struct TcShared {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t mma_fin;
  uint32_t tmem;
  int b, vl, tile;         // where this CTA's range starts
  long long start, end;    // its tiles
  Split split;
  Unfinite unfinite[kUnfinite];
  int32_t par[2][kMaxNodes];
};

// A run of one lane group's tiles in this CTA's range.
struct Seg {
  int b, vl, n, ntiles;  // ntiles: of the whole lane group
  int j0, j1;            // this segment's tiles
};

// Walks the CTA's range segment by segment; every role has its own.
struct Walk {
  int b, vl, tile;
  long long pos, end;
  __device__ __forceinline__ bool next(const Params &p, Seg *s) {
    if (pos >= end) return false;
    while (true) {
      if (b >= p.B) return false;
      s->n = p.seq_lens[b];
      s->ntiles = tiles_of(p, s->n);
      if (s->ntiles > 0) break;
      ++b;  // a refused sequence has no tiles (pos < end: a later one has)
    }
    s->b = b;
    s->vl = vl;
    s->j0 = tile;
    s->j1 = (int)min((long long)s->ntiles, tile + (end - pos));
    pos += s->j1 - s->j0;
    tile = 0;
    if (++vl == p.Hkv * p.MG) {
      vl = 0;
      ++b;
    }
    return true;
  }
};

// Clears this thread's value row of an edge tile in shared memory unless it
// is somebody's (`used`) and finite; true if it was somebody's and was not
// finite.  Starts at chunk (row & 7) of the swizzled row: no bank conflicts.
template <int D>
__device__ __forceinline__ bool clear_value_row(unsigned char *sV, int row, bool used) {
  using K = TcCfg<D, 1>;
  uint32_t odd = 0;
  if (used) {
#pragma unroll
    for (int c = 0; c < K::KB; ++c)
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) {
        const uint4 x = *reinterpret_cast<const uint4 *>(sV + c * K::BLK + row * 128 +
                                                         (((ch + row) & 7) << 4));
        // an exponent of all ones carries into the bit above it
        odd |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
               ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
      }
    odd &= 0x80008000u;
  }
  if (!used || odd) {
#pragma unroll
    for (int c = 0; c < K::KB; ++c)
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
        *reinterpret_cast<uint4 *>(sV + c * K::BLK + row * 128 + (((ch + row) & 7) << 4)) =
            make_uint4(0, 0, 0, 0);
  }
  return odd != 0;
}

// The S buffer of a row tile's kx-th tile, and the phase of that buffer's
// barriers: two buffers taken in turn (NT = 1), or one per row tile.
template <int NT>
__device__ __forceinline__ int s_buffer(int kx, int x) {
  return NT == 1 ? (kx & 1) : x;
}
template <int NT>
__device__ __forceinline__ uint32_t s_phase(int kx) {
  return (uint32_t)(NT == 1 ? (kx >> 1) & 1 : kx & 1);
}

// Whether any of the `threads` softmax threads says so (and a barrier).
__device__ __forceinline__ bool any_of_softmax(bool mine, int threads) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, 3, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)mine), "r"(threads)
      : "memory");
  return r != 0;
}

// The value rows that were cleared for the MMA although they are somebody's:
// adds 2^(s - m) v to this thread's O row (TMEM) where it may read them.
// Warp-wide; rare, so keys and values come from global memory one by one.
template <int D>
__device__ __forceinline__ void add_unfinite(const Params &p, const TcShared &sh, const Seg &sg,
                                             bool mine, int lo, int hi, int lo0, int ncell_tiles,
                                             const Line &line, long long orow, float m_run,
                                             uint32_t tO) {
  const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.q + (mine ? orow : 0) * D;
  const long long ln = (long long)sg.b * p.Hkv + sg.vl / p.MG;
  for (int k = 0; k < kUnfinite; ++k) {
    const int j = sh.unfinite[k].tile;
    if (j < 0) continue;
    const bool draft = j >= ncell_tiles;
    for (int e = 0; e < kTile; ++e) {
      if (!((sh.unfinite[k].bits[e >> 5] >> (e & 31)) & 1u)) continue;
      const int cell = lo0 + j * kTile + e;
      uint32_t word = 0u;
#pragma unroll
      for (int w = 0; w < kMaxNodes / 32; ++w)
        if ((e >> 5) == w) word = line.bits[w];
      const bool reads = mine && (draft ? ((word >> (e & 31)) & 1u) != 0 : cell >= lo && cell < hi);
      const long long at = (draft ? ln * p.t + e : ln * p.C + cell) * D;
      const __nv_bfloat16 *kr = (const __nv_bfloat16 *)(draft ? p.kd : p.k) + at;
      const __nv_bfloat16 *vr = (const __nv_bfloat16 *)(draft ? p.vd : p.v) + at;
      float pe = 0.f;
      if (reads) {
        float s = 0.f;
        for (int c = 0; c < D; ++c) s = fmaf(to_f32(q[c]), to_f32(kr[c]), s);
        pe = exp2f(s * p.scale_log2 - m_run);
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float ov[32];
        tc::tmem_ld32(tO + c * 32, ov);
        tc::tmem_wait_ld();
        if (reads) {
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = fmaf(pe, to_f32(vr[c * 32 + i]), ov[i]);
        }
        __syncwarp();
        tc::tmem_st32(tO + c * 32, ov);
        tc::tmem_wait_st();
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(TcCfg<D, NT>::THREADS, 1)
    rows_splitk_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ CUtensorMap tmKd,
                       const __grid_constant__ CUtensorMap tmVd, const Params p) {
  using K = TcCfg<D, NT>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ TcShared sh;
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int s = 0; s < K::STAGES; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 1);
      mbar_init(&sh.v_full[s], 1);
      mbar_init(&sh.v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.p_full[s], 4);  // a row tile's four warps
      mbar_init(&sh.o_done[s], 1);
      mbar_init(&sh.o_free[s], 4);
    }
    mbar_init(&sh.mma_fin, 1);
    for (int k = 0; k < kUnfinite; ++k) sh.unfinite[k] = Unfinite{-1, {0u, 0u, 0u, 0u}};
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&sh.tmem, kTmemCols);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tmQ);
    tc::prefetch_tmap(&tmK);
    tc::prefetch_tmap(&tmV);
    if (p.tree) {
      tc::prefetch_tmap(&tmKd);
      tc::prefetch_tmap(&tmVd);
    }
  }
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if (warp == 0) {
    // this CTA's range, and the lane group and tile it starts in
    const Split s = split_of(p, lane);
    const long long start = (long long)blockIdx.x * s.per, end = min(s.total, start + s.per);
    const long long LPB = (long long)p.Hkv * p.MG;
    long long cum = 0;
    int b = 0, vl = 0, tile = 0;
    if (start < end) {
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int bb = b0 + lane;
        const long long x = bb < p.B ? tiles_of(p, p.seq_lens[bb]) * LPB : 0;
        long long incl = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, cum + incl > start);
        if (hit) {
          const int src = __ffs(hit) - 1;
          b = b0 + src;
          cum += __shfl_sync(0xffffffffu, incl - x, src);
          const long long nt = __shfl_sync(0xffffffffu, x, src) / LPB;
          vl = (int)((start - cum) / nt);
          tile = (int)((start - cum) - vl * nt);
          break;
        }
        cum += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) {
      sh.b = b;
      sh.vl = vl;
      sh.tile = tile;
      sh.start = start;
      sh.end = end;
      sh.split = s;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  bool failed = false;
  Walk walk{sh.b, sh.vl, sh.tile, sh.start, sh.end};
  Seg sg;

  if (warp >= 4) {
    // ================================================= softmax: one row each
    if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    const int x = (warp - 4) >> 2;           // row tile
    const int q4 = warp & 3;                 // TMEM lane quarter
    const int row = q4 * 32 + lane;          // row within the tile
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tO = tmem + lane_base + K::TM_O + x * D;
    const float sc = p.scale_log2;
    int jj = 0;                              // tiles of the range so far
    int jx = 0;                              // of these, with rows in this row tile
    bool ok = true;
    while (ok && walk.next(p, &sg)) {
      const int g = sg.vl / p.MG, grp = sg.vl - g * p.MG;
      const int rho_x = grp * p.group_rows + x * kM;   // the row tile's first row
      const int nx = min(NT, (p.R - grp * p.group_rows + kM - 1) / kM);  // row tiles here
      if (x >= nx) {  // no rows in this tile: it takes no part in the segment
        jj += sg.j1 - sg.j0;
        continue;
      }
      const int rho = rho_x + row;
      const bool mine = rho < p.R;
      const bool warp_on = rho_x + q4 * 32 < p.R;      // any row of this warp
      const int i = mine ? rho % p.t : 0;
      const int lo0 = first_cell(p, sg.n);
      // what this row may read
      int lo = 0, hi = 0;  // cells [lo, hi)
      Line line;
      line.depth = -1;
#pragma unroll
      for (int w = 0; w < 4; ++w) line.bits[w] = 0u;
      if (p.tree) {
        if (p.parents) {
          // the previous segment's readers are past their masks here
          asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
          if (row < p.t) sh.par[x][row] = p.parents[(long long)sg.b * p.t + row];
          asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
        }
        if (mine) {
          line = line_of(p.parents ? sh.par[x] : nullptr, i, p.window);
          if (line.refused) record_status(p.status, GQA_ERR_TREE);
          if (line.depth >= 0) {
            lo = p.window > 0 ? max(0, sg.n + line.depth - (p.window - 1)) : 0;
            hi = sg.n;
          }
        }
      } else if (mine) {
        hi = sg.n - p.t + i + 1;
      }
      const int ncell_tiles = sg.ntiles - p.tree;
      float m_run = -INFINITY, l_run = 0.f;
      float *srow = p.scores && mine
                        ? p.scores + (((long long)sg.b * p.Hkv + g) * p.R + rho) * p.Cp
                        : nullptr;
      bool found = false;  // value rows cleared that are not finite
      for (int j = sg.j0; j < sg.j1; ++j, ++jj, ++jx) {
        const int sb = s_buffer<NT>(jx, x);
        const bool draft = j >= ncell_tiles;
        const int c0 = lo0 + j * kTile;  // first cell of the tile
        // tiles that some row may not read all of
        const bool edge = draft || c0 + kTile > (p.tree ? sg.n : sg.n - p.t + 1) ||
                          (p.window > 0 && c0 < sg.n + p.t - p.window);
        if (!__all_sync(0xffffffffu, mbar_wait(&sh.s_full[sb], s_phase<NT>(jx), &failed))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t tS = tmem + lane_base + sb * kTile;
        if (warp_on) {
          float s[kTile];
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld32(tS + c * 32, s + c * 32);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kTile; ++e) s[e] *= sc;
          if (edge) {
            if (draft) {
#pragma unroll
              for (int e = 0; e < kTile; ++e)
                if (!((line.bits[e >> 5] >> (e & 31)) & 1u)) s[e] = -INFINITY;
            } else {
              const int a = lo - c0, z = hi - c0;
#pragma unroll
              for (int e = 0; e < kTile; ++e)
                if (e < a || e >= z) s[e] = -INFINITY;
            }
          }
          if (srow) {
#pragma unroll
            for (int e = 0; e < kTile; e += 4)
              *reinterpret_cast<float4 *>(srow + c0 + e) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
          }
          float mc[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < kTile; e += 2) mc[(e >> 1) & 3] = fmax3(mc[(e >> 1) & 3], s[e], s[e + 1]);
          const float m_tile = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
          if (j == sg.j0) {
            m_run = m_tile;
          } else if (__any_sync(0xffffffffu, m_tile > m_run + kLazyRescale)) {
            // O must hold P V of the previous tile before it is rescaled
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.o_done[s_buffer<NT>(jx - 1, x)],
                                                   s_phase<NT>(jx - 1), &failed))) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const float m_new = fmaxf(m_run, m_tile);
            const float alpha = m_new == m_run ? 1.f : exp2f(m_run - m_new);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              float ov[32];
              tc::tmem_ld32(tO + c * 32, ov);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] *= alpha;
              tc::tmem_st32(tO + c * 32, ov);
            }
            tc::tmem_wait_st();
            l_run *= alpha;
            m_run = m_new;
          }
          // bf16 P over the first 64 of S's columns.  The sum takes the fp32
          // values: their roundings to bf16 are independent and average out.
          const float msub = m_run == -INFINITY ? 0.f : m_run;
          float2 lsum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 pv = make_float2(ex2_approx(s[c * 64 + 2 * e] - msub),
                                            ex2_approx(s[c * 64 + 2 * e + 1] - msub));
              lsum = fadd2v(lsum, pv);
              w[e] = __uint_as_float(pack_bf16(pv.x, pv.y));
            }
            tc::tmem_st32(tS + c * 32, w);
          }
          tc::tmem_wait_st();
          l_run += lsum.x + lsum.y;
        }
        if (edge && x == 0) {
          // value rows that some row may not read: row `row` of the V tile
          const int st = jj % K::STAGES;
          const bool vok = mbar_wait(&sh.v_full[st], (jj / K::STAGES) & 1, &failed);
          bool used;
          if (!draft) {
            used = c0 + row < sg.n;
          } else {
            used = row < p.t && (!p.parents || sh.par[0][row] != -2);
          }
          bool odd = false;
          if (vok) odd = clear_value_row<D>(smem + K::OFF_V + st * K::TILE, row, used);
          const uint32_t word = __ballot_sync(0xffffffffu, odd);
          if (word) {  // rare: remember which, for add_unfinite
            found = true;
            if (lane == 0)
              for (int k = 0; k < kUnfinite; ++k) {
                const int was = atomicCAS(&sh.unfinite[k].tile, -1, j);
                if (was == -1 || was == j) {
                  sh.unfinite[k].bits[q4] = word;
                  break;
                }
              }
          }
          tc::fence_proxy_async_smem();
          if (!__all_sync(0xffffffffu, vok)) {
            ok = false;
            break;
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[sb]);
      }
      if (!ok) break;

      // ---- the segment's end: O holds every P V once the last is done
      {
        if (!__all_sync(0xffffffffu, mbar_wait(&sh.o_done[s_buffer<NT>(jx - 1, x)],
                                               s_phase<NT>(jx - 1), &failed))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
      }
      const long long L = (long long)sg.b * p.Hkv * p.MG + sg.vl;
      const bool whole = sg.j0 == 0 && sg.j1 == sg.ntiles;
      const long long slot = L + blockIdx.x;
      const int grow = x * kM + row;  // row within the group
      const long long orow = ((long long)sg.b * p.Hq + (long long)g * p.r) * p.t + rho;
      __nv_bfloat16 *o = (__nv_bfloat16 *)p.o + orow * D;
      float *acc = p.acc + (slot * p.group_rows + grow) * D;
      if (any_of_softmax(found, 128 * nx)) {
        if (warp_on)
          add_unfinite<D>(p, sh, sg, mine, lo, hi, lo0, ncell_tiles, line, orow, m_run, tO);
        any_of_softmax(false, 128 * nx);  // every row has read the list
        if (threadIdx.x == 128)
          for (int k = 0; k < kUnfinite; ++k) sh.unfinite[k] = Unfinite{-1, {0u, 0u, 0u, 0u}};
        any_of_softmax(false, 128 * nx);
      }
      if (mine && p.tree && line.depth < 0) {  // padding, or refused: nothing counts
        m_run = -INFINITY;
        l_run = 0.f;
      }
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      if (warp_on) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float ov[32];
          tc::tmem_ld32(tO + c * 32, ov);
          tc::tmem_wait_ld();
          if (l_run == 0.f) {  // no key at all: zero, whatever the MMA made of it
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = 0.f;
          }
          if (mine && whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w4[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w4[k] = pack_bf16(ov[e * 8 + 2 * k] * inv, ov[e * 8 + 2 * k + 1] * inv);
              *reinterpret_cast<uint4 *>(o + c * 32 + e * 8) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(acc + c * 32 + e) = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
          }
          __syncwarp();
        }
        if (mine && (!whole || p.scores)) p.ml[slot * p.group_rows + grow] = make_float2(m_run, l_run);
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.o_free[x]);
    }
  } else {
    if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      // ================================================= TMA producer
      if (lane == 0) {
        int jj = 0, segs = 0, nk = 0, nv = 0;  // tiles, segments, K and V fills so far
        bool ok = true;
        while (ok && walk.next(p, &sg)) {
          const int g = sg.vl / p.MG, grp = sg.vl - g * p.MG;
          const int nx = min(NT, (p.R - grp * p.group_rows + kM - 1) / kM);
          const int ncell_tiles = sg.ntiles - p.tree, lo0 = first_cell(p, sg.n);
          const int ln = sg.b * p.Hkv + g;
          const int qrow = (sg.b * p.Hq + g * p.r) * p.t + grp * p.group_rows;
          for (int j = sg.j0; ok && j < sg.j1; ++j, ++jj) {
            const int st = jj % K::STAGES;
            const uint32_t par = (jj / K::STAGES - 1) & 1;
            const bool draft = j >= ncell_tiles;
            const CUtensorMap *mk = draft ? &tmKd : &tmK, *mv = draft ? &tmVd : &tmV;
            const int c1 = draft ? 0 : lo0 + j * kTile;
            if (jj >= K::STAGES && !mbar_wait(&sh.k_empty[st], par, &failed)) {
              ok = false;
              break;
            }
            if (j == sg.j0) {
              // Q's buffer is free once the previous segment's last S is done
              if (segs > 0 && !mbar_wait(&sh.q_empty, (segs - 1) & 1, &failed)) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(&sh.q_full, nx * K::TILE);
              for (int xx = 0; xx < nx; ++xx)
#pragma unroll
                for (int c = 0; c < K::KB; ++c)
                  tc::tma_load_2d(smem + xx * K::TILE + c * K::BLK, &tmQ, c * 64, qrow + xx * kM,
                                  &sh.q_full);
              ++segs;
            }
            mbar_arrive_expect_tx(&sh.k_full[st], K::TILE);
#pragma unroll
            for (int c = 0; c < K::KB; ++c)
              tc::tma_load_3d(smem + K::OFF_K + st * K::TILE + c * K::BLK, mk, c * 64, c1, ln,
                              &sh.k_full[st]);
            ++nk;
            if (jj >= K::STAGES && !mbar_wait(&sh.v_empty[st], par, &failed)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sh.v_full[st], K::TILE);
#pragma unroll
            for (int c = 0; c < K::KB; ++c)
              tc::tma_load_3d(smem + K::OFF_V + st * K::TILE + c * K::BLK, mv, c * 64, c1, ln,
                              &sh.v_full[st]);
            ++nv;
          }
        }
        // Never leave a copy in flight into an exiting CTA.
        bool f2 = false;
        if (segs > 0) mbar_wait(&sh.q_full, (segs - 1) & 1, &f2);
        for (int k = max(0, nk - K::STAGES); k < nk; ++k)
          mbar_wait(&sh.k_full[k % K::STAGES], (k / K::STAGES) & 1, &f2);
        for (int k = max(0, nv - K::STAGES); k < nv; ++k)
          mbar_wait(&sh.v_full[k % K::STAGES], (k / K::STAGES) & 1, &f2);
        failed |= f2;
      }
    } else if (warp == 1) {
      // ================================================= MMA issuer
      if (lane == 0) {
        constexpr uint32_t idS = tc::idesc_bf16_f32(kM, kTile, 0, 0);
        constexpr uint32_t idO = tc::idesc_bf16_f32(kM, D, 0, 1);
        int jj = 0, segs = 0;            // tiles and segments of the range so far
        int jx[NT], sx[NT];              // those that row tile x took part in
        for (int xx = 0; xx < NT; ++xx) jx[xx] = sx[xx] = 0;
        bool ok = true;
        // O_x += P_x V of tile k of the range (row tile x's kx-th), `first` of
        // its segment
        auto issue_pv = [&](int k, int xx, int kx, bool first, bool last_x) -> bool {
          const int st = k % K::STAGES;
          const int sb = s_buffer<NT>(kx, xx);
          if (!mbar_wait(&sh.v_full[st], (k / K::STAGES) & 1, &failed)) return false;
          if (!mbar_wait(&sh.p_full[sb], s_phase<NT>(kx), &failed)) return false;
          // the previous segment's O has been read out
          if (first && sx[xx] > 0 && !mbar_wait(&sh.o_free[xx], (sx[xx] - 1) & 1, &failed))
            return false;
          tc::fence_after_sync();
          const uint32_t sV = smem_u32(smem + K::OFF_V + st * K::TILE);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc::mma_bf16_ts(tmem + K::TM_O + xx * D, tmem + sb * kTile + kk * 8,
                            tc::sw128_desc(sV + kk * 16 * 128, K::BLK, 1024), idO,
                            (!first || kk > 0) ? 1u : 0u);
          tc::mma_commit(&sh.o_done[sb]);
          if (last_x) tc::mma_commit(&sh.v_empty[st]);
          return true;
        };
        while (ok && walk.next(p, &sg)) {
          const int grp = sg.vl % p.MG;
          const int nx = min(NT, (p.R - grp * p.group_rows + kM - 1) / kM);
          if (!mbar_wait(&sh.q_full, segs & 1, &failed)) break;
          for (int j = sg.j0; ok && j < sg.j1; ++j, ++jj) {
            const int st = jj % K::STAGES;
            if (!mbar_wait(&sh.k_full[st], (jj / K::STAGES) & 1, &failed)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int xx = 0; xx < NT; ++xx) {
              if (xx >= nx || !ok) continue;
              // NT = 2: S_x(j) overwrites P_x(j-1), so its P V goes first.  NT
              // = 1: S(j) overwrites P(j-2), whose P V was issued already.
              if (NT == 2 && j > sg.j0 &&
                  !issue_pv(jj - 1, xx, jx[xx] - 1, j - 1 == sg.j0, xx == nx - 1)) {
                ok = false;
                continue;
              }
              tc::fence_after_sync();
              const uint32_t sQ = smem_u32(smem + xx * K::TILE);
              const uint32_t sK = smem_u32(smem + K::OFF_K + st * K::TILE);
              const int sb = s_buffer<NT>(jx[xx], xx);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * K::BLK + (kk & 3) * 32;
                tc::mma_bf16_ss(tmem + sb * kTile, tc::sw128_desc(sQ + off, 16, 1024),
                                tc::sw128_desc(sK + off, 16, 1024), idS, kk > 0 ? 1u : 0u);
              }
              tc::mma_commit(&sh.s_full[sb]);
              ++jx[xx];
            }
            if (!ok) break;
            tc::mma_commit(&sh.k_empty[st]);
            if (j + 1 == sg.j1) tc::mma_commit(&sh.q_empty);
            if (NT == 1 && j > sg.j0 && !issue_pv(jj - 1, 0, jx[0] - 2, j - 1 == sg.j0, true))
              ok = false;
          }
#pragma unroll
          for (int xx = 0; xx < NT; ++xx) {
            if (xx >= nx || !ok) continue;
            ok = issue_pv(jj - 1, xx, jx[xx] - 1, sg.j1 - sg.j0 == 1, xx == nx - 1);
            ++sx[xx];
          }
          ++segs;
        }
        // Drain: every MMA has finished before TMEM is freed.
        tc::mma_commit(&sh.mma_fin);
        bool f2 = false;
        mbar_wait(&sh.mma_fin, 0, &f2);
        failed |= f2;
      }
    } else if (warp == 2) {
      // Refused sequences: zero outputs; CTA c takes batch rows c, c + G, ...
      for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (length_ok(p, p.seq_lens[b])) continue;
        if (lane == 0) record_status(p.status, GQA_ERR_CAPACITY);
        uint4 *ob = reinterpret_cast<uint4 *>((__nv_bfloat16 *)p.o + (long long)b * p.Hq * p.t * D);
        for (long long i = lane; i < (long long)p.Hq * p.t * (D / 8); i += 32)
          ob[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }

  if (failed) record_status(p.status, kStatusTimeout);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, kTmemCols);
}

}  // namespace rows
}  // namespace gqa
