// evict.cuh -- eviction from a cache by accumulated attention weight.
//
// Per lane (b, g) of n cells: where n > budget, the last `recent` cells stay
// and, of the cells before them, the budget - recent with the largest
// weights (equal weights: the lowest cell first).  The survivors keep their
// order.  Weights compare by value; -0 equals 0 and NaN is below everything.
//
// evict_select_kernel, one CTA per lane: the weights become ordered 32-bit
// keys, held in registers up to 32 per thread (longer lanes read them again
// from L2).  The k-th largest key T is found digit by digit from the top, 12,
// 10 and 10 bits: a histogram of the digit over the keys that share T's
// higher digits, suffix sums over its bins, the bin that holds rank k.  What
// bounds it is the SM's issue rate, 32768 keys being 1024 warp instructions
// per step of the loop: three passes of one comparison and few additions
// where a search by thresholds takes 16 passes of three comparisons each
// (measured: 8 lanes of 32768 cells 55 us by thresholds of 2 bits).  A warp
// whose lanes agree on a bin adds them at once, so equal weights (zeros, a
// fresh cache) do not queue up on one counter.  A pass that finds exactly k
// keys from T's bin up ends the search.  One prefix sum over (above T, equal
// to T) places every survivor; the CTA writes the list `kept` and its lane's
// weights (read completely before, so they may be compacted in place).
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

constexpr int kBins = 4096;  // of the first, 12-bit digit

// Finds rank k (from the top, 1-based, at most the total count) among the
// bins: the bin that holds it, the count above that bin, its own count.
// Block-wide; BINS is a multiple of kSelThreads.
template <int BINS>
__device__ __forceinline__ void find_bin(const uint32_t *hist, uint32_t k, uint32_t *warp_sum,
                                         uint32_t *result) {
  constexpr int PER = BINS / kSelThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // thread t has bins [BINS - (t + 1) PER, BINS - t PER), from the top down
  uint32_t c[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    c[i] = hist[BINS - 1 - tid * PER - i];
    sum += c[i];
  }
  uint32_t incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint32_t above = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (above < k && k <= above + c[i]) {  // one thread, one bin
      result[0] = BINS - 1 - tid * PER - i;
      result[1] = above;
      result[2] = c[i];
    }
    above += c[i];
  }
  __syncthreads();
}

// KPT > 0: lanes of at most KPT * kSelThreads cells, keys in registers;
// KPT = 0: any length.
template <int KPT>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const Params p) {
  constexpr int STRIPS = KPT > 0 ? KPT : 8;  // strips of kSelThreads cells placed at a time
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t found[3];
  __shared__ uint32_t place[STRIPS * kWarps][2], masks[STRIPS * kWarps][2];
  __shared__ uint32_t wsum[kWarps][2], wtop[kWarps];
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
  // T: the k-th largest candidate key, or after an early end the lower bound
  // of its bin
  uint32_t T = 0, need = 0;  // need: how many of the keys equal to T stay
  bool exact = false;        // every key >= T stays
  if (k > 0) {
    uint32_t rank = k;  // of T among the keys that share its higher digits
#pragma unroll
    for (int pass = 0; pass < 3 && !exact; ++pass) {
      const int shift = pass == 0 ? 20 : (pass == 1 ? 10 : 0);
      const uint32_t low = pass == 0 ? 4095u : 1023u;
      const int upper = shift + (pass == 0 ? 12 : 10);  // bits above the digit are T's
      for (int i = tid; i < (int)low + 1; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      auto count = [&](int j, uint32_t x) {
        const bool in = j < nc && (pass == 0 || (x >> (upper & 31)) == (T >> (upper & 31)));
        const uint32_t bin = (x >> shift) & low;
        const unsigned some = __ballot_sync(0xffffffffu, in);
        if (some == 0) return;
        // the lanes that agree with the first counted one go together
        const int first = __ffs(some) - 1;
        const uint32_t b0 = __shfl_sync(0xffffffffu, bin, first);
        const unsigned same = __ballot_sync(0xffffffffu, in && bin == b0);
        if (lane == first) atomicAdd(&hist[b0], __popc(same));
        if (in && bin != b0) atomicAdd(&hist[bin], 1u);
      };
      if constexpr (KPT > 0) {
#pragma unroll
        for (int i = 0; i < KPT; ++i) count(i * kSelThreads + tid, key[i]);
      } else {
        for (int j0 = 0; j0 < nc; j0 += kSelThreads) {
          const int j = j0 + tid;
          count(j, j < nc ? order_key(w[j]) : 0u);
        }
      }
      __syncthreads();
      if (pass == 0)
        find_bin<4096>(hist, rank, wtop, found);
      else
        find_bin<1024>(hist, rank, wtop, found);
      T |= found[0] << shift;
      rank -= found[1];
      exact = rank == found[2];
    }
    need = rank;  // used when not exact: T is then a key, `rank` of its equals stay
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
      const uint32_t ms = masks[i * kWarps + warp][0], me = masks[i * kWarps + warp][1];
      const bool sure = (ms >> lane) & 1, eq = (me >> lane) & 1;
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
