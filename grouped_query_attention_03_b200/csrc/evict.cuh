// evict.cuh -- eviction from a cache by accumulated attention weight.
//
// Per lane (b, g) of n cells: where n > budget, the last `recent` cells stay
// and, of the cells before them, the budget - recent with the largest
// weights (equal weights: the lowest cell first).  The survivors keep their
// order.  Weights compare by value; -0 equals 0 and NaN is below everything.
//
// evict_select_kernel, one CTA or a cluster of them per lane, each with a run
// of its cells: the weights become ordered 32-bit keys, held in registers (KPT
// per thread; lanes too long for that take one CTA that reads them again from
// L2).  The k-th largest key T is found digit by digit from the top, 11, 11
// and 10 bits: a histogram of the digit over the keys that share T's higher
// digits, added up over the cluster through distributed shared memory;
// suffix sums over its bins and the bin that holds rank k.  A first digit of
// 11 bits (sign, exponent, two more) tells a few dozen magnitudes apart, so
// a warp's keys seldom meet on a counter, and usually the second digit ends
// the search: exactly k keys from T's bin up.  The runs before a CTA's own
// are counted from the same histograms, so one barrier of the cluster per
// digit is all that its CTAs wait for.  One prefix sum over (above T, equal
// to T) places every survivor; the cluster writes the list `kept` and the
// lane's weights (read completely before, so they may be compacted in
// place).  Bound by latency: reading the weights, counting and scanning each
// digit, the cluster's barriers and remote counts, placing.
//
// Moving the rows is a gather through `kept`, bound by bandwidth (64 lanes of
// 8000 cells to 4096, 273 MB: 56.4 us with the selection, of 41.7 at the copy
// rate).  Into other caches any order will do: evict_copy_kernel.  In
// place, destinations are at or below their sources but rows of other
// chunks may still be unread, so a CTA owns a column slice of a lane's K or
// V and walks the rows in ascending order, a chunk loaded completely before
// it is stored and the next chunk's loads already in flight (they read at or
// above their own destinations, which are above everything stored so far).
// Column slices never meet, so this needs no waiting between CTAs (64 lanes of
// 8000 cells to 4096: 66 us with the selection, of 42 at the copy rate; 8 of 32768
// to 4096, 64 CTAs: 27 of 5.5).
#pragma once

#include "common.cuh"

namespace gqa {
namespace evict {

constexpr int kSelThreads = 512;
constexpr int kWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kPB = kBins / kSelThreads;  // bins per thread

struct Params {
  const float *w;
  float *w_out;
  const int32_t *seq_lens;
  int32_t *lens_out, *kept, *status;
  int B, Hkv, C, C_out, budget, recent;
};

// Ascending order of the weights as unsigned integers; NaN is 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The weight of a key (every NaN comes back as one NaN).
__device__ __forceinline__ float key_weight(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four words of shared memory at the same place in CTA `rank` of the cluster.
__device__ __forceinline__ uint4 ld_cluster4(const uint32_t *at, uint32_t rank) {
  uint32_t addr;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(at)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// KPT > 0: a CTA's run is at most KPT * kSelThreads cells, keys in registers;
// KPT = 0: any length, a cluster of one CTA.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const Params p, int cluster) {
  constexpr int STRIPS = KPT > 0 ? KPT : 8;  // strips of kSelThreads cells placed at a time
  static_assert(kPB == 4, "a thread's bins are one 16-byte read");
  __shared__ __align__(16) uint32_t hist[2][kBins];  // [digit & 1], bins from the top down
  __shared__ uint32_t wtop[kWarps], wbase[kWarps][2], found[3];
  __shared__ uint32_t place[STRIPS * kWarps][2], masks[STRIPS * kWarps][2];
  __shared__ uint32_t wsum[kWarps][2];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t L = blockIdx.x / cluster;
  const int rank = (int)(blockIdx.x - L * cluster);
  const int b = (int)(L / p.Hkv);
  const float *w = p.w + L * p.C;
  float *wo = p.w_out + L * p.C_out;
  int32_t *kept = p.kept + L * p.budget;
  const int t0 = rank * kSelThreads + tid, step = cluster * kSelThreads;
  // this CTA's cells [r0, r1): whole strips of the capacity, so that the
  // weights are on their way before the length is known
  const int run = (p.C + cluster * kSelThreads - 1) / (cluster * kSelThreads) * kSelThreads;
  const int r0 = min(p.C, rank * run);
  uint32_t key[STRIPS];
  if constexpr (KPT > 0) {
    float x[KPT];
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int j = r0 + i * kSelThreads + tid;
      x[i] = i * kSelThreads < run && j < p.C ? w[j] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < KPT; ++i) key[i] = order_key(x[i]);
  }
  const int n = p.seq_lens[b];
  if (n < 0 || n > p.C) {  // (the same for the whole cluster)
    if (t0 == 0) record_status(p.status, GQA_ERR_CAPACITY);
    for (int i = t0; i < p.budget; i += step) kept[i] = -1;
    return;
  }
  if (n <= p.budget) {  // nothing leaves
    for (int i = t0; i < p.budget; i += step) kept[i] = i < n ? i : -1;
    if (wo != w)
      for (int i = t0; i < n; i += step) wo[i] = w[i];
    for (int i = n + t0; i < p.C_out; i += step) wo[i] = 0.f;
    return;
  }
  const int nc = n - p.recent;             // candidates: cells [0, nc)
  const uint32_t k = p.budget - p.recent;  // of which the k heaviest stay; k <= nc
  const int r1 = min(n, r0 + run);
  // T: the k-th largest candidate key, or after an early end the lower bound
  // of its bin
  uint32_t T = 0, need = 0;  // need: how many of the keys equal to T stay
  bool exact = false;        // every key >= T stays
  // survivors for sure and keys equal to T in the runs before this one; the
  // recent cells among them stay
  uint32_t base_s = max(0, min(r0, n) - nc), base_e = 0;
  if (k > 0) {
    uint32_t rank_k = k;  // of T among the keys that share its higher digits
    for (int pass = 0; pass < 3 && !exact; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t low = pass < 2 ? 2047u : 1023u;
      const int above_bits = pass == 0 ? 0 : (pass == 1 ? 21 : 10);  // shift that leaves the higher digits
      uint32_t *h = hist[pass & 1];
      *reinterpret_cast<uint4 *>(h + tid * kPB) = make_uint4(0, 0, 0, 0);
      __syncthreads();
      auto count = [&](int j, uint32_t x) {
        if (j < r1 && j < nc && (pass == 0 || (x >> above_bits) == (T >> above_bits)))
          atomicAdd(&h[kBins - 1 - ((x >> shift) & low)], 1u);
      };
      if constexpr (KPT > 0) {
#pragma unroll
        for (int i = 0; i < KPT; ++i) count(r0 + i * kSelThreads + tid, key[i]);
      } else {
        for (int j = r0 + tid; j < r1; j += kSelThreads) count(j, order_key(w[j]));
      }
      // this thread's four bins: over the cluster, and over the runs before
      uint4 c, before = make_uint4(0, 0, 0, 0);
      if (cluster > 1) {
        // (the others read this histogram until the next digit's barrier, and
        // the next digit has the other one)
        cluster_sync();
        c = make_uint4(0, 0, 0, 0);
        for (int r = 0; r < cluster; ++r) {
          if (r == rank) before = c;
          const uint4 y = ld_cluster4(h + tid * kPB, r);
          c.x += y.x;
          c.y += y.y;
          c.z += y.z;
          c.w += y.w;
        }
      } else {
        __syncthreads();
        c = *reinterpret_cast<const uint4 *>(h + tid * kPB);
      }
      const uint32_t cc[4] = {c.x, c.y, c.z, c.w}, cb[4] = {before.x, before.y, before.z, before.w};
      const uint32_t sum = c.x + c.y + c.z + c.w;
      uint32_t incl = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      if (lane == 31) wtop[warp] = incl;
      __syncthreads();
      uint32_t above = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? wtop[lane] : 0u);
      const uint32_t my_above = above;
#pragma unroll
      for (int i = 0; i < kPB; ++i) {
        if (above < rank_k && rank_k <= above + cc[i]) {  // one thread, one bin
          found[0] = kBins - 1 - (tid * kPB + i);
          found[1] = above;
          found[2] = cc[i];
        }
        above += cc[i];
      }
      __syncthreads();
      T |= found[0] << shift;
      const uint32_t up = found[1];
      exact = rank_k - up == found[2];
      if (cluster > 1) {
        // of the runs before: keys in bins above the found one, and in it
        uint32_t bs = 0, be = 0, at = my_above;
#pragma unroll
        for (int i = 0; i < kPB; ++i) {
          if (at + cc[i] <= up) bs += cb[i];  // above (empty bins hold nothing)
          if (kBins - 1 - (tid * kPB + i) == (int)found[0]) be = cb[i];
          at += cc[i];
        }
        bs = __reduce_add_sync(0xffffffffu, bs);
        be = __reduce_add_sync(0xffffffffu, be);
        if (lane == 0) {
          wbase[warp][0] = bs;
          wbase[warp][1] = be;
        }
        __syncthreads();
        base_s += __reduce_add_sync(0xffffffffu, lane < kWarps ? wbase[lane][0] : 0u);
        base_e = __reduce_add_sync(0xffffffffu, lane < kWarps ? wbase[lane][1] : 0u);
      }
      rank_k -= up;
    }
    need = rank_k;  // used when not exact: T is then a key, `need` of its equals stay
    if (exact) {    // the keys in T's bin stay too
      base_s += base_e;
      base_e = 0;
    }
  }
  if (cluster > 1) {
    if (k == 0) cluster_sync();  // every weight of the lane has been read
    // nobody leaves before all have read its counts: waited for at the end
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  // does cell j (of key kk) stay for sure, or as one of the equal ones?
  auto sure_of = [&](int j, uint32_t kk) {
    return j < r1 && (j >= nc || (k > 0 && (exact ? kk >= T : kk > T)));
  };
  auto equal_of = [&](int j, uint32_t kk) { return j < r1 && j < nc && k > 0 && !exact && kk == T; };
  // Place the survivors, STRIPS * kSelThreads cells at a time in ascending
  // order: cell -> strip, warp, lane.
  for (int s0 = r0; s0 < r1; s0 += STRIPS * kSelThreads) {
    if constexpr (KPT == 0) {
#pragma unroll
      for (int i = 0; i < STRIPS; ++i) {
        const int j = s0 + i * kSelThreads + tid;
        key[i] = j < r1 ? order_key(w[j]) : 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < STRIPS; ++i) {
      const int j = s0 + i * kSelThreads + tid;
      const uint32_t ms = __ballot_sync(0xffffffffu, sure_of(j, key[i]));
      const uint32_t me = __ballot_sync(0xffffffffu, equal_of(j, key[i]));
      if (lane == 0) {
        place[i * kWarps + warp][0] = __popc(ms);
        place[i * kWarps + warp][1] = __popc(me);
        masks[i * kWarps + warp][0] = ms;
        masks[i * kWarps + warp][1] = me;
      }
    }
    __syncthreads();
    // exclusive prefix sums over the STRIPS * kWarps (<= kSelThreads) counts
    uint32_t es = 0, ee = 0, is, ie;
    if (tid < STRIPS * kWarps) {
      es = place[tid][0];
      ee = place[tid][1];
    }
    is = es;
    ie = ee;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, is, off), c = __shfl_up_sync(0xffffffffu, ie, off);
      if (lane >= off) {
        is += x;
        ie += c;
      }
    }
    if (lane == 31) {
      wsum[warp][0] = is;
      wsum[warp][1] = ie;
    }
    __syncthreads();
    const bool in_w = lane < kWarps;
    const uint32_t s_l = in_w ? wsum[lane][0] : 0u, e_l = in_w ? wsum[lane][1] : 0u;
    const uint32_t ws = __reduce_add_sync(0xffffffffu, lane < warp ? s_l : 0u);
    const uint32_t we = __reduce_add_sync(0xffffffffu, lane < warp ? e_l : 0u);
    const uint32_t ts = __reduce_add_sync(0xffffffffu, s_l), te = __reduce_add_sync(0xffffffffu, e_l);
    if (tid < STRIPS * kWarps) {
      place[tid][0] = base_s + ws + is - es;
      place[tid][1] = base_e + we + ie - ee;
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < STRIPS; ++i) {
      const int j = s0 + i * kSelThreads + tid;
      const uint32_t ms = masks[i * kWarps + warp][0], me = masks[i * kWarps + warp][1];
      const bool sure = (ms >> lane) & 1, eq = (me >> lane) & 1;
      const uint32_t s = place[i * kWarps + warp][0] + __popc(ms & below);
      const uint32_t e = place[i * kWarps + warp][1] + __popc(me & below);
      if (sure || (eq && e < need)) {
        const uint32_t at = s + min(e, need);
        kept[at] = j;
        // in place: at <= j, and every weight up to this strip has been read
        // before the barriers above (of all runs, with a cluster)
        wo[at] = key_weight(key[i]);
      }
    }
    base_s += ts;
    base_e += te;
    __syncthreads();
  }
  for (int i = p.budget + t0; i < p.C_out; i += step) wo[i] = 0.f;
  if (cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// New lengths, written where the moves are launched (the selection has read
// the old ones).
__device__ __forceinline__ void write_lengths(const Params &p) {
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int n = p.seq_lens[b];
    p.lens_out[b] = (n < 0 || n > p.C) ? n : min(n, p.budget);
  }
}

// Into other caches: every vector of every kept row, in any order.
template <typename V>
__global__ void __launch_bounds__(256)
    evict_copy_kernel(const V *__restrict__ kc, const V *__restrict__ vc, V *__restrict__ ko,
                      V *__restrict__ vo, const Params p, int vpr) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if (blockIdx.x == 0) write_lengths(p);
  constexpr int U = 4;
  const int64_t total = (int64_t)p.B * p.Hkv * p.budget * vpr;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i0 < total; i0 += U * stride) {
    V x[U], y[U];
    int64_t dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * stride;
      dst[u] = -1;
      if (i >= total) continue;
      const int64_t row = i / vpr, lane = row / p.budget;
      const int e = (int)(i - row * vpr), at = (int)(row - lane * p.budget);
      const int j = p.kept[row];
      if (j < 0) continue;
      const int64_t src = (lane * p.C + j) * vpr + e;
      dst[u] = (lane * p.C_out + at) * vpr + e;
      x[u] = kc[src];
      y[u] = vc[src];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (dst[u] >= 0) {
        ko[dst[u]] = x[u];
        vo[dst[u]] = y[u];
      }
  }
}

// In place: CTA = (lane, K or V, slice of SL vectors of the row).
template <typename V, int SL>
__global__ void __launch_bounds__(256)
    evict_move_kernel(V *kc, V *vc, const Params p, int vpr, int slices) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if (blockIdx.x == 0) write_lengths(p);
  constexpr int U = 8, ROWS = 256 / SL;
  const int64_t lane = (int64_t)blockIdx.x / (2 * slices);
  const int rest = (int)(blockIdx.x - lane * 2 * slices);
  const int col = (rest >> 1) * SL + threadIdx.x % SL;
  V *cache = ((rest & 1) ? vc : kc) + lane * p.C * vpr + col;
  const int32_t *kept = p.kept + lane * p.budget;
  const int r0 = threadIdx.x / SL;
  const bool on = col < vpr;
  V x[2][U];
  int src[2][U];
  auto load = [&](int s, int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * ROWS + r0;
      const int j = (on && i < p.budget) ? kept[i] : -1;
      src[s][u] = j > i ? j : -1;  // unmoved rows need nothing
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[s][u] >= 0) x[s][u] = cache[(int64_t)src[s][u] * vpr];
  };
  load(0, 0);
  for (int i0 = 0; i0 < p.budget; i0 += 2 * U * ROWS) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int i = i0 + s * U * ROWS;
      load(s ^ 1, i + U * ROWS);
      __syncthreads();  // this chunk's rows have all been read
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (src[s][u] >= 0) cache[(int64_t)(i + u * ROWS + r0) * vpr] = x[s][u];
    }
  }
}

}  // namespace evict
}  // namespace gqa
