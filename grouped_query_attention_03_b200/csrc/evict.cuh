// evict.cuh -- eviction from a cache by accumulated attention weight.
//
// Per lane (b, g) of n cells: where n > budget, the last `recent` cells stay
// and, of the cells before them, the budget - recent with the largest
// weights (equal weights: the lowest cell first).  The survivors keep their
// order.  Weights compare by value; -0 equals 0 and NaN is below everything.
//
// evict_select_kernel, one CTA per lane: the weights become ordered 32-bit
// keys held in registers (KPT per thread; longer lanes read them again from
// L2 every round).  The largest threshold T that at least k keys reach is
// built from its top bits, two bits per round: each round counts the keys
// that reach the three candidates, so 16 rounds of compares and one block
// reduction find the k-th largest key exactly, whatever the distribution,
// with no atomics (a histogram's would meet on the few bins that weights of
// one magnitude share).  A round ends the search early when exactly k keys
// reach its threshold.  One prefix sum over (above T, equal to T) places
// every survivor; the CTA writes the list `kept` and its lane's weights
// (read completely before, so they may be compacted in place).
//
// Moving the rows (evict_move_kernel) is a gather through `kept`, bound by
// bandwidth.  Into other caches any order will do: evict_copy_kernel.  In
// place, destinations are at or below their sources but rows of other
// chunks may still be unread, so a CTA owns a column slice of a lane's K or
// V and walks the rows in ascending order, a chunk loaded completely before
// it is stored and the next chunk's loads already in flight (they read at or
// above their own destinations, which are above everything stored so far).
// Column slices never meet, so this needs no waiting between CTAs.
#pragma once

#include "common.cuh"

namespace gqa {
namespace evict {

constexpr int kSelThreads = 1024;
constexpr int kWarps = kSelThreads / 32;

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

// Sums (a, b, c) over the block; every thread gets them.  `buf` alternates
// between two halves so that one barrier per call is enough.
__device__ __forceinline__ void block_sum3(uint32_t &a, uint32_t &b, uint32_t &c,
                                           uint32_t (*buf)[3][kWarps], int &turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = __reduce_add_sync(0xffffffffu, a);
  b = __reduce_add_sync(0xffffffffu, b);
  c = __reduce_add_sync(0xffffffffu, c);
  if (lane == 0) {
    buf[turn][0][warp] = a;
    buf[turn][1][warp] = b;
    buf[turn][2][warp] = c;
  }
  __syncthreads();
  a = __reduce_add_sync(0xffffffffu, buf[turn][0][lane]);
  b = __reduce_add_sync(0xffffffffu, buf[turn][1][lane]);
  c = __reduce_add_sync(0xffffffffu, buf[turn][2][lane]);
  turn ^= 1;
}

// KPT > 0: lanes of at most KPT * kSelThreads cells, keys in registers;
// KPT = 0: any length.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const Params p) {
  constexpr int STRIPS = KPT > 0 ? KPT : 8;  // strips of kSelThreads cells placed at a time
  __shared__ uint32_t sums[2][3][kWarps];
  __shared__ uint32_t place[STRIPS * kWarps][2];
  __shared__ uint32_t wsum[kWarps][2];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t L = blockIdx.x;
  const int b = (int)(L / p.Hkv);
  const int n = p.seq_lens[b];
  const float *w = p.w + L * p.C;
  float *wo = p.w_out + L * p.C_out;
  int32_t *kept = p.kept + L * p.budget;
  if (n < 0 || n > p.C) {
    if (tid == 0) record_status(p.status, GQA_ERR_CAPACITY);
    for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = -1;
    return;
  }
  if (n <= p.budget) {  // nothing leaves
    for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = i < n ? i : -1;
    if (wo != w)
      for (int i = tid; i < n; i += kSelThreads) wo[i] = w[i];
    for (int i = n + tid; i < p.C_out; i += kSelThreads) wo[i] = 0.f;
    return;
  }
  const int nc = n - p.recent;          // candidates: cells [0, nc)
  const uint32_t k = p.budget - p.recent;  // of which the k heaviest stay; k <= nc
  uint32_t key[STRIPS];
  if constexpr (KPT > 0) {
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int j = i * kSelThreads + tid;
      key[i] = j < n ? order_key(w[j]) : 0u;
    }
  }
  // T: the k-th largest candidate key; `more` candidates are above T - or,
  // after an early end, T is any threshold that exactly k reach
  uint32_t T = 0, need = 0;  // need: how many of the keys equal to T stay
  bool exact = false;        // every key >= T stays
  int turn = 0;
  if (k > 0) {
    for (int bit = 30; bit >= 0 && !exact; bit -= 2) {
      const uint32_t t1 = T | (1u << bit), t2 = T | (2u << bit), t3 = T | (3u << bit);
      uint32_t c1 = 0, c2 = 0, c3 = 0;
      auto count = [&](int j, uint32_t x) {
        if (j < nc) {
          c1 += x >= t1;
          c2 += x >= t2;
          c3 += x >= t3;
        }
      };
      if constexpr (KPT > 0) {
#pragma unroll
        for (int i = 0; i < KPT; ++i) count(i * kSelThreads + tid, key[i]);
      } else {
        for (int j = tid; j < nc; j += kSelThreads) count(j, order_key(w[j]));
      }
      block_sum3(c1, c2, c3, sums, turn);
      uint32_t c = 0;
      if (c3 >= k) { T = t3; c = c3; }
      else if (c2 >= k) { T = t2; c = c2; }
      else if (c1 >= k) { T = t1; c = c1; }
      exact = c == k;
    }
    if (!exact) {
      uint32_t above = 0, z0 = 0, z1 = 0;
      if constexpr (KPT > 0) {
#pragma unroll
        for (int i = 0; i < KPT; ++i) above += (i * kSelThreads + tid < nc) && key[i] > T;
      } else {
        for (int j = tid; j < nc; j += kSelThreads) above += order_key(w[j]) > T;
      }
      block_sum3(above, z0, z1, sums, turn);
      need = k - above;
    }
  }
  // Place the survivors, STRIPS * kSelThreads cells at a time in ascending
  // order: cell -> strip, warp, lane.
  uint32_t base_s = 0, base_e = 0;  // survivors for sure, keys equal to T, so far
  for (int s0 = 0; s0 < n; s0 += STRIPS * kSelThreads) {
    if constexpr (KPT == 0) {
#pragma unroll
      for (int i = 0; i < STRIPS; ++i) {
        const int j = s0 + i * kSelThreads + tid;
        key[i] = j < n ? order_key(w[j]) : 0u;
      }
    }
    // does cell j (of key kk) stay for sure, or as one of the equal ones?
    auto sure_of = [&](int j, uint32_t kk) {
      return j < n && (j >= nc || (k > 0 && (exact ? kk >= T : kk > T)));
    };
    auto equal_of = [&](int j, uint32_t kk) { return j < nc && k > 0 && !exact && kk == T; };
#pragma unroll
    for (int i = 0; i < STRIPS; ++i) {
      const int j = s0 + i * kSelThreads + tid;
      const uint32_t ms = __ballot_sync(0xffffffffu, sure_of(j, key[i]));
      const uint32_t me = __ballot_sync(0xffffffffu, equal_of(j, key[i]));
      if (lane == 0) {
        place[i * kWarps + warp][0] = __popc(ms);
        place[i * kWarps + warp][1] = __popc(me);
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
      const uint32_t a = __shfl_up_sync(0xffffffffu, is, off), c = __shfl_up_sync(0xffffffffu, ie, off);
      if (lane >= off) {
        is += a;
        ie += c;
      }
    }
    if (lane == 31) {
      wsum[warp][0] = is;
      wsum[warp][1] = ie;
    }
    __syncthreads();
    uint32_t ws = lane < warp ? wsum[lane][0] : 0u, we = lane < warp ? wsum[lane][1] : 0u;
    uint32_t ts = wsum[lane][0], te = wsum[lane][1];
    ws = __reduce_add_sync(0xffffffffu, ws);
    we = __reduce_add_sync(0xffffffffu, we);
    ts = __reduce_add_sync(0xffffffffu, ts);
    te = __reduce_add_sync(0xffffffffu, te);
    if (tid < STRIPS * kWarps) {
      place[tid][0] = base_s + ws + is - es;
      place[tid][1] = base_e + we + ie - ee;
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < STRIPS; ++i) {
      const int j = s0 + i * kSelThreads + tid;
      const bool sure = sure_of(j, key[i]), eq = equal_of(j, key[i]);
      const uint32_t ms = __ballot_sync(0xffffffffu, sure);
      const uint32_t me = __ballot_sync(0xffffffffu, eq);
      const uint32_t s = place[i * kWarps + warp][0] + __popc(ms & below);
      const uint32_t e = place[i * kWarps + warp][1] + __popc(me & below);
      if (sure || (eq && e < need)) {
        const uint32_t at = s + min(e, need);
        kept[at] = j;
        // in place: at <= j, and every weight of this and earlier strips has
        // been read before the barriers above
        wo[at] = key_weight(key[i]);
      }
    }
    base_s += ts;
    base_e += te;
    __syncthreads();
  }
  for (int i = p.budget + tid; i < p.C_out; i += kSelThreads) wo[i] = 0.f;
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
