// rows_splitk.cuh -- tcgen05/TMEM split-K attention of a KV group's query rows
// over a cache: gqa_decode_tree and gqa_decode_scored for bf16 with d = 64 or
// 128 (sm_100a).  Which keys a row reads, the split over CTAs and
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
//   warps 4-11  softmax.  NT = 1: two warpgroups, each with 64 of a tile's
//               128 keys, a thread per row, with its own running maximum, sum
//               and O, combined once at the end of a segment; NT = 2: a
//               warpgroup per row tile, a thread per row with all 128 keys.
//               A thread loads its scores, masks edge tiles, rescales O when
//               its maximum grew by more than 2^8 and writes bf16 P over S;
//               at the end of a segment the O row goes out (a lane group in
//               one part) or to the workspace.
// TMEM: NT = 1 has two S buffers, so S(j+1) is computed under the softmax of
// tile j, and two O; NT = 2 has one S and one O per row tile, and the two
// take turns.
//
// Bound by HBM with one row tile: a 128-key tile is 4 d * 128 bytes, 1.5 us of
// an SM's share of the bandwidth at d = 128 (8 sequences of 8000 cells, 26
// nodes, 32 heads on 8: 57 us, 4.7 TB/s, of which 11 us start and end; 48 ragged
// sequences to 4000, 16 nodes: 83 us, of 65 at the copy rate; the same with d =
// 64, where a tile's masks and softmax are as long as at 128: 72 of 32).  Two
// row tiles take about 2.3 us per 128 keys (1.1 PFLOP/s), each tile's products
// and softmax in turn with the other's; short segments then show what a
// segment costs besides its tiles, 7 to 9 us of masks, queries and O's way out
// (64 ragged sequences, 63 nodes, 8 heads on 1: 104 us, 0.65 PFLOP/s).
// P enters its product as bf16, since V is (the tensor cores take both operands
// in one type): one rounding of at most 2^-8 per weight, independent of each
// other, so an output is off by 2.3e-3 in relative L2 where its own rounding
// alone makes 1.6e-3; the rows' sums, and what cells received, are of the fp32
// weights.  The remainders as a second bf16 operand would take a second P V.
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
constexpr int kTcThreads = 384;
// Registers per thread after the split: 128 * low + 256 * high must not exceed
// the 384 threads times the 168 they are launched with.  The softmax warps
// would use more: the compiler spills 142 (NT = 1) to 280 bytes (NT = 2) a
// thread, which the times above include.
constexpr int kRegsLow = 72, kRegsHigh = 216;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= 384 * 168, "register split");
constexpr int kAddParts = 4;               // parts a CTA adds to its own O at most
constexpr int kUnfinite = 4;               // edge tiles of a segment at most

template <int D, int NT>
struct TcCfg {
  static constexpr int NC = NT == 1 ? 64 : 128;  // keys of a tile per softmax thread
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
  static_assert(TM_O + 2 * D <= kTmemCols, "S and O must fit in TMEM");
};

struct Unfinite {  // value rows of one edge tile cleared for the MMA
  int tile;
  uint32_t bits[4];
};

// A lane group in several parts: its first part's CTA and their number.
struct Group {
  long long L;
  int c0, np;
};
struct TcShared {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2], o_done[2], o_free[2];
  uint64_t p_full[2][2];   // [S buffer][key half]: P of these 64 keys written
  uint64_t mma_fin;
  uint64_t early_full, early_done;  // the first segment's part: written, counted
  uint32_t tmem;
  int b, vl, off;          // where this CTA's range starts
  long long start, end;    // its tiles
  long long per;           // positions of every CTA
  int pad, aligned;        // (see Split)
  int early_last;             // that part was its group's last
  Group late;                 // the last segment's group, to be merged
  int32_t len[kLenCache];
  Unfinite unfinite[kUnfinite];
  int32_t par[2][kMaxNodes];
};

// A run of one lane group's tiles in this CTA's range.
struct Seg {
  long long first;       // where the lane group's first tile is, over all CTAs
  int b, vl, n, ntiles;  // ntiles: of the whole lane group
  int j0, j1;            // this segment's tiles
};

__device__ __forceinline__ Group group_of(const Params &p, const Seg &sg, long long per) {
  Group r;
  r.L = (long long)sg.b * p.Hkv * p.MG + sg.vl;
  r.c0 = (int)udiv(sg.first, per);
  r.np = (int)udiv(sg.first + sg.ntiles - 1, per) - r.c0 + 1;
  return r;
}
// The first segment, when it ends a lane group that began in an earlier CTA
// and others follow: its part is counted as soon as it is written.
__device__ __forceinline__ bool is_early(const Params &p, const Seg &sg, bool first, bool more) {
  return !p.finish && first && more && sg.j0 > 0;
}

// Walks the CTA's range segment by segment; every role has its own.
struct Walk {
  int b, vl, off;          // off: into the lane group's extent, pad first
  int pad, aligned;
  long long pos, end;
  const int32_t *cached;   // the lengths in shared memory
  __device__ __forceinline__ bool next(const Params &p, Seg *s) {
    while (true) {
      if (pos >= end || b >= p.B) return false;
      s->n = b < kLenCache ? cached[b] : p.seq_lens[b];
      s->ntiles = tiles_of(p, s->n);
      if (s->ntiles > 0) {
        const int skip = max(0, pad - off);
        pos += skip;
        off += skip;
        break;
      }
      ++b;  // a refused sequence has no tiles
      vl = 0;
    }
    if (pos >= end) return false;
    s->b = b;
    s->vl = vl;
    s->j0 = off - pad;
    s->first = pos - s->j0;
    s->j1 = (int)min((long long)s->ntiles, s->j0 + (end - pos));
    pos += s->j1 - s->j0;
    off = 0;
    if (aligned) pos = end;  // one group per CTA
    if (++vl == p.Hkv * p.MG) {
      vl = 0;
      ++b;
    }
    return true;
  }
};

// Where this CTA's range starts.  Warp-wide; the first kLenCache lengths are
// left in `cache`.
struct Start {
  int b, vl, off;
  long long pos, end;
  Split split;
};
__device__ __forceinline__ Start start_of(const Params &p, int lane, int32_t *cache) {
  const Split s = split_of(p, lane, cache);
  Start r{0, 0, 0, (long long)blockIdx.x * s.per, 0, s};
  r.end = min(s.total, r.pos + s.per);
  if (r.pos >= r.end) return r;
  const long long LPB = (long long)p.Hkv * p.MG;
  long long cum = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int bb = b0 + lane;
    const long long x =
        bb < p.B ? extent_of(p, s, bb < kLenCache ? cache[bb] : __ldcg(p.seq_lens + bb)) * LPB : 0;
    long long incl = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, cum + incl > r.pos);
    if (hit) {
      const int src = __ffs(hit) - 1;
      r.b = b0 + src;
      cum += __shfl_sync(0xffffffffu, incl - x, src);
      const long long ext = udiv(__shfl_sync(0xffffffffu, x, src), LPB);
      r.vl = (int)udiv(r.pos - cum, ext);
      r.off = (int)((r.pos - cum) - r.vl * ext);
      return r;
    }
    cum += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// The bits below position k (k <= 0: none, k >= 32: all).
__device__ __forceinline__ uint32_t below(int k) {
  return k >= 32 ? 0xffffffffu : (1u << max(k, 0)) - 1u;
}

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

__device__ __forceinline__ uint64_t l2_policy_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// tma_load_3d with an L2 cache policy.
__device__ __forceinline__ void tma_load_3d_hint(void *smem_dst, const CUtensorMap *map, int c0,
                                                 int c1, int c2, uint64_t *bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)),
      "l"(policy)
      : "memory");
}

// Two 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st2(uint32_t taddr, float a, float b) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b))
               : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, float &a, float &b) {
  uint32_t x, y;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];"
               : "=r"(x), "=r"(y)
               : "r"(taddr));
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}

// Whether any of the `threads` softmax threads says so (and a barrier).  The
// end of the kernel has a barrier of its own: the second warpgroup may be
// there while the first is still in a segment that is its alone; and so has
// such a segment (the first warpgroup's, 1), since a second warpgroup whose
// wait ran out may be in a later one.
// These barriers have no limit of their own.  They end because every warp
// that takes part in one always comes to it: a warp whose wait ran out (its
// later waits then return at once) skips its work and its arrivals, but walks
// on through the same segments and barriers as the others, whose number
// depends on nothing but the split and on what they agree on at a barrier.
constexpr int kBarSegment = 3, kBarEnd = 4;
__device__ __forceinline__ bool any_of_softmax(bool mine, int threads, int bar = kBarSegment) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, %3, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)mine), "r"(threads), "r"(bar)
      : "memory");
  return r != 0;
}

// The value rows that were cleared for the MMA although they are somebody's:
// adds 2^(s - m) v to this thread's O row (TMEM) where it may read them, for
// keys [e_first, e_last) of the tiles.
// Warp-wide; rare, so keys and values come from global memory one by one.
template <int D>
__device__ __forceinline__ void add_unfinite(const Params &p, const TcShared &sh, const Seg &sg,
                                             bool mine, int lo, int hi, int lo0, int ncell_tiles,
                                             const Line &line, long long orow, float m_run,
                                             uint32_t tO, int e_first, int e_last) {
  const __nv_bfloat16 *q = (const __nv_bfloat16 *)p.q + (mine ? orow : 0) * D;
  const long long ln = (long long)sg.b * p.Hkv + sg.vl / p.MG;
  for (int k = 0; k < kUnfinite; ++k) {
    const int j = sh.unfinite[k].tile;
    if (j < 0) continue;
    const bool draft = j >= ncell_tiles;
    for (int e = e_first; e < e_last; ++e) {
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

// 32 columns of this thread's O: NT = 1 combines the two halves' (a0, a1).
// Zero without keys, whatever the MMA made of it.
template <int D, int NT>
__device__ __forceinline__ void load_o(uint32_t taddr, float a0, float a1, bool none, float *ov) {
  tc::tmem_ld32(taddr, ov);
  if constexpr (NT == 1) {
    float ow[32];
    tc::tmem_ld32(taddr + D, ow);
    tc::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) ov[e] = none ? 0.f : ov[e] * a0 + ow[e] * a1;
  } else {
    tc::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) ov[e] = none ? 0.f : ov[e];
  }
}

__device__ __forceinline__ int ld_acquire_gpu(const int *p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Merges a lane group's parts and writes its rows: the 256 softmax threads,
// through the K and V rings.
template <int D>
__device__ __forceinline__ void merge_group(const Params &p, const Group &gr, unsigned char *smem,
                                         int warp) {
  const long long ln = gr.L / p.MG;
  const int grp = (int)(gr.L - ln * p.MG);
  const int rows = min(p.group_rows, p.R - grp * p.group_rows);
  const long long row0 = ln * p.R + (long long)grp * p.group_rows;
  float *tile = reinterpret_cast<float *>(smem);
  constexpr int pitch = D + 4;
  merge_parts<8>(p, gr.L + gr.c0, gr.np, rows, warp, tile, pitch, p.lse ? p.lse + row0 : nullptr);
  any_of_softmax(false, 256, kBarEnd);
  __nv_bfloat16 *o = (__nv_bfloat16 *)p.o + row0 * D;
  for (int e = (threadIdx.x - 128) * 8; e < rows * D; e += 256 * 8) {
    const float *src = tile + (e / D) * pitch + e % D;
    *reinterpret_cast<uint4 *>(o + e) =
        make_uint4(pack_bf16(src[0], src[1]), pack_bf16(src[2], src[3]), pack_bf16(src[4], src[5]),
                   pack_bf16(src[6], src[7]));
  }
  any_of_softmax(false, 256, kBarEnd);
}

template <int D, int NT>
__global__ void __launch_bounds__(kTcThreads, 1)
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
      mbar_init(&sh.p_full[s][0], 4);  // a warpgroup's four warps
      mbar_init(&sh.p_full[s][1], 4);
      mbar_init(&sh.o_done[s], 1);
      mbar_init(&sh.o_free[s], NT == 1 ? 8 : 4);  // the warps that read O_x
    }
    mbar_init(&sh.mma_fin, 1);
    mbar_init(&sh.early_full, 8);
    mbar_init(&sh.early_done, 1);
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
    const Start at = start_of(p, lane, sh.len);
    if (lane == 0) {
      sh.b = at.b;
      sh.vl = at.vl;
      sh.off = at.off;
      sh.start = at.pos;
      sh.end = at.end;
      sh.per = at.split.per;
      sh.pad = at.split.pad;
      sh.aligned = at.split.aligned;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  bool failed = false;
  Walk walk{sh.b, sh.vl, sh.off, sh.pad, sh.aligned, sh.start, sh.end, sh.len};
  Seg sg;

  if (warp >= 4) {
    // ================================================= softmax: one row each
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    constexpr int NC = K::NC;
    const int wg = (warp - 4) >> 2;          // warpgroup
    const int x = NT == 1 ? 0 : wg;          // row tile
    const int e0 = NT == 1 ? wg * NC : 0;    // first key of a tile
    const int q4 = warp & 3;                 // TMEM lane quarter
    const int row = q4 * 32 + lane;          // row within the row tile
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tO = tmem + lane_base + K::TM_O + wg * D;
    // Scores are compared as they come and scaled in the exponent's FMA; a
    // negative scale turns the order around, and 0 is a scale too small to
    // show.  A masked score is the infinity that the scale makes negative.
    const float sc = p.scale_log2 == 0.f ? 1e-30f : p.scale_log2;
    const bool neg = sc < 0.f;
    const float masked = neg ? INFINITY : -INFINITY;
    bool first_seg = true;
    int left = 0;                            // the last segment's part was left behind
    int was_b = -1, was_grp = -1;            // whose masks `line`, lo, hi are
    // the parent of node `row` in this sequence and, ahead of time, the next
    const int32_t *parents = p.tree ? p.parents : nullptr;
    int par_b = walk.b, par_next = -2;
    if (parents && row < p.t && par_b < p.B) par_next = parents[(long long)par_b * p.t + row];
    int lo = 0, hi = 0;                      // cells [lo, hi) this row may read
    Line line;
    line.depth = -1;
#pragma unroll
    for (int w = 0; w < 4; ++w) line.bits[w] = 0u;
    int jj = 0;                              // tiles of the range so far
    int jx = 0;                              // of these, with rows in this row tile
    // `failed` is the same for a warp's lanes wherever it is looked at
    while (walk.next(p, &sg)) {  // (a warp that gave up walks on: see any_of_softmax)
      const int g = sg.vl / p.MG, grp = sg.vl - g * p.MG;
      const int rho_x = grp * p.group_rows + x * kM;   // the row tile's first row
      const int nx = min(NT, (p.R - grp * p.group_rows + kM - 1) / kM);  // row tiles here
      const bool more = walk.pos < walk.end;           // segments may follow
      const bool is_e = is_early(p, sg, first_seg, more);
      first_seg = false;
      if (x >= nx) {  // no rows in this tile: it takes no part in the segment
        jj += sg.j1 - sg.j0;
        if (is_e && lane == 0) mbar_arrive(&sh.early_full);
        continue;
      }
      const int rho = rho_x + row;
      const bool mine = rho < p.R;
      const bool warp_on = rho_x + q4 * 32 < p.R;      // any row of this warp
      const int lo0 = first_cell(p, sg.n);
      // what this row may read: the same for all lanes of a sequence
      if (sg.b != was_b || grp != was_grp) {
        const int i = mine ? rho % p.t : 0;
        lo = hi = 0;
        if (p.tree) {
          if (p.parents && sg.b != was_b) {
            // the previous segment's readers are past their masks here
            asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
            if (row < p.t)
              sh.par[wg][row] = sg.b == par_b ? par_next : parents[(long long)sg.b * p.t + row];
            asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
            par_b = sg.b + 1;
            if (row < p.t && par_b < p.B) par_next = parents[(long long)par_b * p.t + row];
          }
          if (mine) {
            line = line_of(p.parents ? sh.par[wg] : nullptr, i, p.window);
            if (line.refused) record_status(p.status, GQA_ERR_TREE);
            if (line.depth >= 0) {
              lo = p.window > 0 ? max(0, sg.n + line.depth - (p.window - 1)) : 0;
              hi = sg.n;
            }
          }
        } else if (mine) {
          hi = sg.n - p.t + i + 1;
        }
        was_b = sg.b;
        was_grp = grp;
      }
      const int ncell_tiles = sg.ntiles - p.tree;
      float m_run = -INFINITY, l_run = 0.f;
      float *srow = p.scores && mine
                        ? p.scores + (((long long)sg.b * p.Hkv + g) * p.R + rho) * p.Cp + e0
                        : nullptr;
      bool found = false;  // value rows cleared that are not finite
      int j = sg.j0;
      for (; !failed && j < sg.j1; ++j, ++jj, ++jx) {
        const int sb = s_buffer<NT>(jx, x);
        const bool draft = j >= ncell_tiles;
        const int c0 = lo0 + j * kTile;  // first cell of the tile
        // tiles that some row may not read all of
        const bool edge = draft || c0 + kTile > (p.tree ? sg.n : sg.n - p.t + 1) ||
                          (p.window > 0 && c0 < sg.n + p.t - p.window);
        if (!__all_sync(0xffffffffu, mbar_wait(&sh.s_full[sb], s_phase<NT>(jx), &failed))) {
          failed = true;
          break;
        }
        tc::fence_after_sync();
        if (edge && (NT == 1 ? (q4 >> 1) == wg : wg == 0)) {
          // value rows that some row may not read: row `row` of the V tile
          // (NT = 1: by the warps of its own key half)
          const int st = jj % K::STAGES;
          const bool vok = mbar_wait(&sh.v_full[st], (jj / K::STAGES) & 1, &failed);
          // cells behind the sequence and padding are nobody's; of the others,
          // finite or not matters only where some row may not read them
          const bool used = draft ? row < p.t && (!p.parents || sh.par[wg][row] != -2)
                                  : c0 + row < sg.n;
          const bool all_read = p.tree && !draft && !(p.window > 0 && c0 < sg.n + p.t - p.window);
          bool odd = false;
          if (vok && !(used && all_read))
            odd = clear_value_row<D>(smem + K::OFF_V + st * K::TILE, row, used);
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
            failed = true;
            break;
          }
        }
        const uint32_t tS = tmem + lane_base + sb * kTile + e0;
        if (!warp_on) {  // no rows: nothing to write, but counted
          if (lane == 0) {
            mbar_arrive(&sh.p_full[sb][NT == 1 ? wg : 0]);
            if (NT == 2) mbar_arrive(&sh.p_full[sb][1]);
          }
        } else {
          float s[NC];
#pragma unroll
          for (int c = 0; c < NC / 32; ++c) tc::tmem_ld32(tS + c * 32, s + c * 32);
          tc::tmem_wait_ld();
          if (edge) {
            // the tile's keys that this row reads, as bits
#pragma unroll
            for (int w = 0; w < NC / 32; ++w) {
              uint32_t bits;
              if (draft)
                bits = NT == 1 ? (wg ? line.bits[2 + w] : line.bits[w]) : line.bits[w];
              else
                bits = below(hi - c0 - e0 - 32 * w) & ~below(lo - c0 - e0 - 32 * w);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(bits & (1u << e))) s[w * 32 + e] = masked;
            }
          }
          if (srow) {
#pragma unroll
            for (int e = 0; e < NC; e += 4)
              *reinterpret_cast<float4 *>(srow + c0 + e) =
                  make_float4(s[e] * sc, s[e + 1] * sc, s[e + 2] * sc, s[e + 3] * sc);
          }
          float mx;
          {
            float mc[4] = {masked, masked, masked, masked};
            if (!neg) {
#pragma unroll
              for (int e = 0; e < NC; e += 2) mc[(e >> 1) & 3] = fmax3(mc[(e >> 1) & 3], s[e], s[e + 1]);
              mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
            } else {
#pragma unroll
              for (int e = 0; e < NC; ++e) mc[e & 3] = fminf(mc[e & 3], s[e]);
              mx = fminf(fminf(mc[0], mc[1]), fminf(mc[2], mc[3]));
            }
          }
          const float m_tile = mx * sc;  // -inf where every score is masked
          if (j == sg.j0) {
            m_run = m_tile;
          } else if (__any_sync(0xffffffffu, m_tile > m_run + kLazyRescale)) {
            // O must hold P V of the previous tile before it is rescaled
            if (!__all_sync(0xffffffffu, mbar_wait(&sh.o_done[s_buffer<NT>(jx - 1, x)],
                                                   s_phase<NT>(jx - 1), &failed))) {
              failed = true;
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
          // bf16 P over the first half of this thread's S columns.  The sum
          // takes the fp32 values: their roundings to bf16 are independent
          // and average out.
          const float msub = m_run == -INFINITY ? 0.f : m_run;
          const float2 sc2 = make_float2(sc, sc), nm2 = make_float2(-msub, -msub);
          float2 lsum = make_float2(0.f, 0.f);
          // published 64 keys at a time: the P V of the first half starts under
          // the exponentials of the second (NT = 2)
#pragma unroll
          for (int c = 0; c < NC / 64; ++c) {
            float w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 v = ffma2v(make_float2(s[c * 64 + 2 * e], s[c * 64 + 2 * e + 1]), sc2, nm2);
              const float2 pv = make_float2(ex2_approx(v.x), ex2_approx(v.y));
              lsum = fadd2v(lsum, pv);
              w[e] = __uint_as_float(pack_bf16(pv.x, pv.y));
            }
            tc::tmem_st32(tS + c * 32, w);
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[sb][NT == 1 ? wg : c]);
          }
          l_run += lsum.x + lsum.y;
        }
      }
      jj += sg.j1 - j;  // (0 but after a wait that ran out)
      jx += sg.j1 - j;

      // ---- the segment's end: O holds every P V once the last is done
      if (!failed && !__all_sync(0xffffffffu, mbar_wait(&sh.o_done[s_buffer<NT>(jx - 1, x)],
                                                   s_phase<NT>(jx - 1), &failed)))
        failed = true;
      tc::fence_after_sync();
      const bool whole = sg.j0 == 0 && sg.j1 == sg.ntiles;
      const int grow = x * kM + row;  // row within the group
      const long long orow = ((long long)sg.b * p.Hq + (long long)g * p.r) * p.t + rho;
      const int parties = NT == 1 ? 256 : 128 * nx;
      const int bar = parties == 256 ? kBarSegment : 1;
      const bool works = !failed && warp_on;
      if (any_of_softmax(found, parties, bar)) {
        if (works)
          add_unfinite<D>(p, sh, sg, mine, lo, hi, lo0, ncell_tiles, line, orow, m_run, tO, e0, e0 + NC);
        any_of_softmax(false, parties, bar);  // every row has read the list
        if (threadIdx.x == 128)
          for (int k = 0; k < kUnfinite; ++k) sh.unfinite[k] = Unfinite{-1, {0u, 0u, 0u, 0u}};
        any_of_softmax(false, parties, bar);
      }
      // NT = 1: the halves swap (m, l); each thread then combines d / 2
      // columns of both O: o = O_0 a_0 + O_1 a_1, a_h = 2^(m_h - max)
      float m_all = m_run, l_all = l_run, a0 = 1.f, a1 = 0.f;
      if constexpr (NT == 1) {
        // through the unused columns behind P in the last tile's S buffer.
        // The next segment's first S goes to the other buffer; its second
        // comes to this one, and the MMA lane holds it back until every warp
        // is through here (o_free).
        const uint32_t tX = tmem + lane_base + s_buffer<NT>(jx - 1, x) * kTile + 32;
        if (!failed) {
          tmem_st2(tX + wg * 64, m_run, l_run);
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        any_of_softmax(false, parties, bar);
        tc::fence_after_sync();
        float m0 = -INFINITY, l0 = 0.f, m1 = -INFINITY, l1 = 0.f;
        if (!failed) {
          tmem_ld2(tX, m0, l0);
          tmem_ld2(tX + 64, m1, l1);
          tc::tmem_wait_ld();
        }
        m_all = fmaxf(m0, m1);
        // (a half whose scores are all NaN has m = -inf and keeps its NaN sum)
        a0 = m0 == m_all ? 1.f : exp2f(m0 - m_all);
        a1 = m1 == m_all ? 1.f : exp2f(m1 - m_all);
        l_all = l0 * a0 + l1 * a1;
      }
      if (p.tree && line.depth < 0) {  // padding, or refused: nothing counts
        m_all = -INFINITY;
        l_all = 0.f;
      }
      // A part that is not the whole group goes to the workspace and is
      // counted, the early one by warp 3.  A last segment's part whose fellows
      // have all been counted, before or after its own, needs no merge: this
      // CTA adds theirs to its O (up to kAddParts of them).
      constexpr int OC = NT == 1 ? D / 2 : D;  // columns this thread writes
      const int oc0 = NT == 1 ? wg * OC : 0;
      const uint32_t tOa = tmem + lane_base + K::TM_O + (NT == 1 ? oc0 : x * D);
      const Group gr = group_of(p, sg, sh.per);
      if (p.finish && sg.j0 == 0 && threadIdx.x == 128) p.groups[gr.L] = make_int2(gr.c0, gr.np);
      bool add = false;
      // (aligned groups' parts end together: looking first would be too early)
      if (!whole && !is_e && !p.finish && !sh.aligned && gr.np <= kAddParts) {
        bool all = false;
        if (threadIdx.x == 128) all = ld_acquire_gpu(&p.counters[gr.c0]) == gr.np - 1;
        add = any_of_softmax(all, parties, bar);
        if (add && threadIdx.x == 128) p.counters[gr.c0] = 0;
      }
      if (!whole && !add) {
        // partials as [column / 4][row][4]: a warp's 32 rows are 512 bytes
        if (works) {
          float4 *acc = reinterpret_cast<float4 *>(p.acc) +
                        ((gr.L + blockIdx.x) * (D / 4) + oc0 / 4) * p.group_rows + grow;
#pragma unroll 1
          for (int c = 0; c < OC / 32; ++c) {
            float ov[32];
            load_o<D, NT>(tOa + c * 32, a0, a1, l_all == 0.f, ov);
            if (mine) {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                acc[(long long)(c * 8 + e / 4) * p.group_rows] =
                    make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
            }
            __syncwarp();
          }
          if (mine && (NT == 2 || wg == 0))
            p.ml[(gr.L + blockIdx.x) * p.group_rows + grow] = make_float2(m_all, l_all);
          __syncwarp();
        }
        if (is_e) {
          if (!failed && lane == 0) mbar_arrive(&sh.early_full);
        } else if (!p.finish) {
          any_of_softmax(false, parties, bar);  // the part is written
          bool last = false;
          if (!failed && threadIdx.x == 128) last = count_part(&p.counters[gr.c0], gr.np);
          add = any_of_softmax(last, parties, bar);
          if (add && gr.np > kAddParts) {
            add = false;
            left = 1;
            if (threadIdx.x == 128) sh.late = gr;
          }
        }
      }
      if ((whole || add) && works) {
        const float2 *ml = p.ml + (gr.L + gr.c0) * p.group_rows + min(grow, p.group_rows - 1);
        const int me = (int)blockIdx.x - gr.c0;
        float m_out = m_all, l_out = l_all;
        if (add) {  // the exact maximum, then the terms in order
          float2 y[kAddParts];
#pragma unroll
          for (int k = 0; k < kAddParts; ++k)
            y[k] = k < gr.np && k != me ? __ldcg(&ml[(long long)k * p.group_rows])
                                        : make_float2(m_all, k == me ? l_all : 0.f);
#pragma unroll
          for (int k = 0; k < kAddParts; ++k) m_out = fmaxf(m_out, y[k].x);
          l_out = 0.f;
#pragma unroll
          for (int k = 0; k < kAddParts; ++k) l_out = fmaf(part_weight(y[k], m_out), y[k].y, l_out);
        }
        const float inv = l_out == 0.f ? 0.f : 1.f / l_out;  // 0: no key at all
        __nv_bfloat16 *o = (__nv_bfloat16 *)p.o + orow * D + oc0;
        const float4 *acc = reinterpret_cast<const float4 *>(p.acc) +
                            ((gr.L + gr.c0) * (D / 4) + oc0 / 4) * p.group_rows +
                            min(grow, p.group_rows - 1);
#pragma unroll 1
        for (int c = 0; c < OC / 32; ++c) {
          float ov[32];
          load_o<D, NT>(tOa + c * 32, a0, a1, l_all == 0.f, ov);
          if (add) {
            float a[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] = 0.f;
#pragma unroll 1
            for (int k = 0; k < gr.np; ++k) {
              if (k == me) {
                const float w = part_weight(make_float2(m_all, l_all), m_out);
#pragma unroll
                for (int e = 0; e < 32; ++e) a[e] = fmaf(w, ov[e], a[e]);
              } else {
                float4 v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  v[e] = __ldcg(&acc[((long long)k * (D / 4) + c * 8 + e) * p.group_rows]);
                const float w = part_weight(__ldcg(&ml[(long long)k * p.group_rows]), m_out);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  a[4 * e] = fmaf(w, v[e].x, a[4 * e]);
                  a[4 * e + 1] = fmaf(w, v[e].y, a[4 * e + 1]);
                  a[4 * e + 2] = fmaf(w, v[e].z, a[4 * e + 2]);
                  a[4 * e + 3] = fmaf(w, v[e].w, a[4 * e + 3]);
                }
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = a[e];
          }
          if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w4[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w4[k] = pack_bf16(ov[e * 8 + 2 * k] * inv, ov[e * 8 + 2 * k + 1] * inv);
              *reinterpret_cast<uint4 *>(o + c * 32 + e * 8) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          }
          __syncwarp();
        }
        if (p.lse && mine && (NT == 2 || wg == 0))
          p.lse[((long long)sg.b * p.Hkv + g) * p.R + rho] =
              make_float2(m_out == -INFINITY ? 0.f : m_out, inv);
        __syncwarp();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (!failed && lane == 0) mbar_arrive(&sh.o_free[x]);
    }
    // Groups whose last part was counted here and could not be added above
    // are merged from the workspace, through the rings, which are empty by
    // now: every tile has been multiplied.  (The first warpgroup takes part in
    // every segment and speaks for both.)
    if (any_of_softmax(!failed && left, 256, kBarEnd)) merge_group<D>(p, sh.late, smem, warp - 4);
    Walk begin{sh.b, sh.vl, sh.off, sh.pad, sh.aligned, sh.start, sh.end, sh.len};
    if (begin.next(p, &sg) && is_early(p, sg, true, begin.pos < begin.end)) {
      if (!__all_sync(0xffffffffu, mbar_wait(&sh.early_done, 0, &failed))) failed = true;
      if (any_of_softmax(!failed && sh.early_last, 256, kBarEnd))
        merge_group<D>(p, group_of(p, sg, sh.per), smem, warp - 4);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      // ================================================= TMA producer
      if (lane == 0) {
        // Q's tiles of the segment.  The first segment's go ahead of its keys;
        // later ones wait for the buffer (the previous segment's last S), and
        // their first keys and values do not wait with them.
        auto load_q = [&](int seg, int nx, int row0, int ln) -> bool {
          if (seg > 0 && !mbar_wait(&sh.q_empty, (seg - 1) & 1, &failed)) return false;
          mbar_arrive_expect_tx(&sh.q_full, nx * K::TILE);
          for (int xx = 0; xx < nx; ++xx)
#pragma unroll
            for (int c = 0; c < K::KB; ++c)
              tc::tma_load_3d(smem + xx * K::TILE + c * K::BLK, &tmQ, c * 64, row0 + xx * kM, ln,
                              &sh.q_full);
          return true;
        };
        // a single pass over the cache evicts itself first, so that parts and
        // outputs stay in L2; with several groups per lane others read it too.
        // (Scored rows' keys are read a second time, by another kernel, and
        // leave all the same.)
        const uint64_t once = p.MG == 1 ? tc::l2_policy_evict_first() : l2_policy_normal();
        int jj = 0, segs = 0, nk = 0, nv = 0;  // tiles, segments, K and V fills so far
        bool ok = true;
        while (ok && walk.next(p, &sg)) {
          const int g = sg.vl / p.MG, grp = sg.vl - g * p.MG;
          const int nx = min(NT, (p.R - grp * p.group_rows + kM - 1) / kM);
          const int ncell_tiles = sg.ntiles - p.tree, lo0 = first_cell(p, sg.n);
          const int ln = sg.b * p.Hkv + g;
          const int row0 = grp * p.group_rows;
          if (segs == 0 && load_q(0, nx, row0, ln)) segs = 1;
          const bool q_due = jj > 0;
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
            mbar_arrive_expect_tx(&sh.k_full[st], K::TILE);
#pragma unroll
            for (int c = 0; c < K::KB; ++c)
              tma_load_3d_hint(smem + K::OFF_K + st * K::TILE + c * K::BLK, mk, c * 64, c1, ln,
                               &sh.k_full[st], once);
            ++nk;
            if (jj >= K::STAGES && !mbar_wait(&sh.v_empty[st], par, &failed)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sh.v_full[st], K::TILE);
#pragma unroll
            for (int c = 0; c < K::KB; ++c)
              tma_load_3d_hint(smem + K::OFF_V + st * K::TILE + c * K::BLK, mv, c * 64, c1, ln,
                               &sh.v_full[st], once);
            ++nv;
            if (j == sg.j0 && q_due) {
              ok = load_q(segs, nx, row0, ln);
              segs += ok;
            }
          }
        }
        // Never leave a copy in flight into an exiting CTA: each that was
        // asked for is waited for, whatever became of the others.
        auto landed = [&](uint64_t *bar, int parity) {
          bool late = false;
          mbar_wait(bar, parity, &late);
          failed |= late;
        };
        if (segs > 0) landed(&sh.q_full, (segs - 1) & 1);
        for (int k = max(0, nk - K::STAGES); k < nk; ++k)
          landed(&sh.k_full[k % K::STAGES], (k / K::STAGES) & 1);
        for (int k = max(0, nv - K::STAGES); k < nv; ++k)
          landed(&sh.v_full[k % K::STAGES], (k / K::STAGES) & 1);
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
          // the previous segment's O has been read out
          if (first && sx[xx] > 0 && !mbar_wait(&sh.o_free[xx], (sx[xx] - 1) & 1, &failed))
            return false;
          const uint32_t sV = smem_u32(smem + K::OFF_V + st * K::TILE);
          // 64 keys at a time, as their P is written: NT = 1 into the half's
          // own O, NT = 2 both into the row tile's
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!mbar_wait(&sh.p_full[sb][h], s_phase<NT>(kx), &failed)) return false;
            tc::fence_after_sync();
            // P's first column: over the half's own scores, or behind each other
            const uint32_t tP = tmem + sb * kTile + h * (NT == 1 ? 64 : 32);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_bf16_ts(tmem + K::TM_O + (NT == 1 ? h : xx) * D, tP + kk * 8,
                              tc::sw128_desc(sV + (h * 4 + kk) * 16 * 128, K::BLK, 1024), idO,
                              (!first || kk > 0 || (NT == 2 && h > 0)) ? 1u : 0u);
          }
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
            // NT = 1: the second tile's S goes where the previous segment's
            // softmax warps exchange their (m, l).  (They read no S before they
            // are through with that, so nobody waits longer than before.)
            if (NT == 1 && j == sg.j0 + 1 && sx[0] > 0 &&
                !mbar_wait(&sh.o_free[0], (sx[0] - 1) & 1, &failed)) {
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
    } else if (lane == 0) {
      // ================================================= warp 3: the early part
      if (walk.next(p, &sg) && is_early(p, sg, true, walk.pos < walk.end)) {
        int last = 0;
        if (mbar_wait(&sh.early_full, 0, &failed)) {
          const Group gr = group_of(p, sg, sh.per);
          last = count_part(&p.counters[gr.c0], gr.np) ? 1 : 0;
        }
        sh.early_last = last;
        mbar_arrive(&sh.early_done);
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
