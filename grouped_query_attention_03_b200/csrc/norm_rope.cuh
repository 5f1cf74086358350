// norm_rope.cuh -- norms of queries and keys for each head, with the
// position rotation in the same pass.
//
// The rows of one projection, [B,T,(Hq + 2 Hkv) d] (query heads, key heads,
// value heads), become the head-major q [B,Hq,T,d], k and v [B,Hkv,T,d] that
// the attention entry points take.  For a query or key head's row x:
//   y = x / sqrt(mean(x^2) + eps) * w                     (where w is given)
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a)      for pair i of y,
//   a = positions[axis(i)][b,t] * inv_freq[i],
// pair i being elements (i, i + rot/2) or (2i, 2i + 1); elements from rot on
// are not rotated, value rows are copied.  All of it in fp32, rounded once.
//
// Angles.  Only the angle's fraction of a turn matters, and a far position
// times a frequency has far more whole turns than fp32 has bits.  Per pair
// F = frac(inv_freq / 2 pi) as a 64-bit fixed-point fraction (one fp64
// product); position * F in wrapping 64-bit integers IS the fraction of the
// angle, exact up to the 2^-53 of F: the error is below |position| * 2^-54
// turns, and the top 32 bits go to sincospif as a signed half turn in
// [-1, 1).
//
// Bound by bandwidth: each element read and written once, 8-10 flops.
// vec kernel: a group of G = 8, 16 or 32 lanes owns a token and a range of
// heads; a lane holds 16 bytes of a row, so the row's sum of squares and the
// other half of each pair are a few shuffles away, and each lane's sines
// and cosines, multiplied into the weights once, serve all its heads.  The
// groups of a CTA own consecutive tokens: a head's output rows are written
// as one run.  generic kernel: any width and alignment, a warp per row
// through shared memory.
#pragma once

#include "common.cuh"

namespace gqa {
namespace nr {

constexpr int kMaxAxes = 4;
constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // head rows a group has in flight

struct Params {
  const void *qkv, *qw, *kw;
  const float *inv_freq;
  const int32_t *positions;  // [axes,B,T] or NULL (position t)
  void *q, *k, *v;
  int64_t batch_stride, row_stride;  // elements
  int64_t tokens;                    // B * T
  int Hq, Hkv, T, d, half, interleaved;
  int hpg, chunks;  // heads per group, groups per token
  float eps, inv_d;
  uint32_t axis[8];  // pair i's axis in bits 2 (i % 16) of word i / 16
};

// frac(f / 2 pi) * 2^64; the quotient's whole turns are dropped first.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  constexpr double kInv2Pi = 0.15915494309189533577;
  const double t = (double)f * kInv2Pi;
  return (uint64_t)((t - floor(t)) * 18446744073709551616.0);
}

// The position of token `tok` (b * T + t) that pair i turns by.
__device__ __forceinline__ int position_of(const Params &p, int64_t tok, int i) {
  if (!p.positions) return (int)(tok % p.T);
  const int ax = (p.axis[i >> 4] >> (2 * (i & 15))) & 3;
  return p.positions[ax * p.tokens + tok];
}

__device__ __forceinline__ void angle(const Params &p, int64_t tok, int i, float *sn, float *cs) {
  const uint64_t frac = (uint64_t)(int64_t)position_of(p, tok, i) * turn_fraction(p.inv_freq[i]);
  sincospif((float)(int32_t)(frac >> 32) * 4.656612873077393e-10f, sn, cs);  // 2^-31
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float *x) {
    x[0] = bf16lo_to_f32(u.x); x[1] = bf16hi_to_f32(u.x);
    x[2] = bf16lo_to_f32(u.y); x[3] = bf16hi_to_f32(u.y);
    x[4] = bf16lo_to_f32(u.z); x[5] = bf16hi_to_f32(u.z);
    x[6] = bf16lo_to_f32(u.w); x[7] = bf16hi_to_f32(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 u, float *x) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};

// 16 bytes, streamed: every row is read once and every output written once.
__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Rows of d elements as d / N vectors on G lanes (the last lanes idle when
// d / N is not a power of two).  Needs 16-byte-aligned rows and, for the
// (i, i + half) pairing, half a multiple of N, so that a lane's partners
// are the same places of one other lane's vector.
template <typename T, int G>
__global__ void __launch_bounds__(kThreads) norm_rope_vec_kernel(const Params p) {
  constexpr int N = Vec<T>::N;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int gl = threadIdx.x % G;  // lane of the group
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
  // every group of the warp takes part in its shuffles, its own unit or not
  const bool mine = unit < p.tokens * p.chunks;
  const int64_t tok = mine ? unit % p.tokens : 0;
  const int chunk = mine ? (int)(unit / p.tokens) : 0;
  const int64_t b = tok / p.T, t = tok - b * p.T;
  const int e0 = gl * N;  // first element of this lane
  const bool on = mine && e0 < p.d;
  const int hn = p.Hq + p.Hkv;
  const int h_first = chunk * p.hpg, h_last = min(h_first + p.hpg, hn + p.Hkv);
  const T *src = (const T *)p.qkv + b * p.batch_stride + t * p.row_stride + e0;

  uint4 raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    raw[u] = (on && h_first + u < h_last) ? ld_stream(src + (int64_t)(h_first + u) * p.d)
                                          : make_uint4(0, 0, 0, 0);

  // this lane's cosines and signed sines, and where its partners are
  const int hv = p.half / N;  // lanes from one half to the other
  const bool lowhalf = gl < hv;
  const int partner =
      (p.interleaved || gl >= 2 * hv) ? gl : (lowhalf ? gl + hv : gl - hv);
  float cs[N], sn[N];
#pragma unroll
  for (int i = 0; i < N; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
  if (on && h_first < hn) {
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        if (e0 + i < 2 * p.half) {
          angle(p, tok, (e0 + i) / 2, &sn[i + 1], &cs[i]);
          sn[i] = -sn[i + 1];
          cs[i + 1] = cs[i];
        }
      }
    } else if (gl < 2 * hv) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        angle(p, tok, (lowhalf ? e0 : e0 - p.half) + i, &sn[i], &cs[i]);
        if (lowhalf) sn[i] = -sn[i];
      }
    }
  }
  // y_e = r (x_e A_e + x_partner(e) B_e),  A = w cos, B = +-w_partner sin,
  // r = 1 / sqrt(mean + eps): rebuilt where the heads change from Q to K
  float A[N], Bc[N];
  auto weigh = [&](const T *w) {
    const int pe0 = partner * N;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pe = p.interleaved ? (e0 + (i ^ 1)) : pe0 + i;
      A[i] = cs[i] * (w && on ? to_f32(w[e0 + i]) : 1.f);
      Bc[i] = sn[i] * (w && on ? to_f32(w[pe]) : 1.f);
    }
  };
  bool norm = false;
  const unsigned full = 0xffffffffu;
  for (int h0 = 0; h0 < p.hpg; h0 += kUnroll) {
    uint4 next[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h_first + h0 + kUnroll + u;
      next[u] = (on && h0 + kUnroll < p.hpg && h < h_last) ? ld_stream(src + (int64_t)h * p.d)
                                                           : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h_first + h0 + u;
      if (h0 + u >= p.hpg) break;  // the same for every lane
      if ((h0 == 0 && u == 0) || h == p.Hq) {
        const T *w = (const T *)(h < p.Hq ? p.qw : p.kw);
        norm = w != nullptr;
        if (h < hn) weigh(w);
      }
      uint4 out = raw[u];
      // a warp's groups may be at different heads (its tokens wrap into the
      // next chunk), so the shuffles run for value rows too
      float x[N], y[N];
      Vec<T>::unpack(raw[u], x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int off = G / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(full, ss, off);
      float xp[N];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < N; ++i) xp[i] = x[i ^ 1];
      } else {
        uint4 o;
        o.x = __shfl_sync(full, raw[u].x, partner, G);
        o.y = __shfl_sync(full, raw[u].y, partner, G);
        o.z = __shfl_sync(full, raw[u].z, partner, G);
        o.w = __shfl_sync(full, raw[u].w, partner, G);
        Vec<T>::unpack(o, xp);
      }
      if (h < hn) {
        const float r = norm ? rsqrtf(fmaf(ss, p.inv_d, p.eps)) : 1.f;
#pragma unroll
        for (int i = 0; i < N; ++i)  // past rot there is no partner (and inf * 0 is not 0)
          y[i] = (e0 + i < 2 * p.half ? fmaf(x[i], A[i], xp[i] * Bc[i]) : x[i] * A[i]) * r;
        out = Vec<T>::pack(y);
      }
      if (on && h < h_last) {
        T *dst;
        if (h < p.Hq)
          dst = (T *)p.q + ((b * p.Hq + h) * p.T + t) * p.d;
        else if (h < hn)
          dst = (T *)p.k + ((b * p.Hkv + (h - p.Hq)) * p.T + t) * p.d;
        else
          dst = (T *)p.v + ((b * p.Hkv + (h - hn)) * p.T + t) * p.d;
        *reinterpret_cast<uint4 *>(dst + e0) = out;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) raw[u] = next[u];
  }
}

// Any width up to GQA_MAX_HEAD_DIM, any alignment: a warp per row.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_row_kernel(const Params p) {
  __shared__ float rows[kThreads / 32][GQA_MAX_HEAD_DIM];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.Hq + 2 * p.Hkv, hn = p.Hq + p.Hkv;
  float *row = rows[warp];
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + warp; w < p.tokens * H; w += stride) {
    const int64_t tok = w / H;
    const int h = (int)(w - tok * H);
    const int64_t b = tok / p.T, t = tok - b * p.T;
    const T *src = (const T *)p.qkv + b * p.batch_stride + t * p.row_stride + (int64_t)h * p.d;
    T *dst;
    if (h < p.Hq)
      dst = (T *)p.q + ((b * p.Hq + h) * p.T + t) * p.d;
    else if (h < hn)
      dst = (T *)p.k + ((b * p.Hkv + (h - p.Hq)) * p.T + t) * p.d;
    else
      dst = (T *)p.v + ((b * p.Hkv + (h - hn)) * p.T + t) * p.d;
    if (h >= hn) {
      for (int e = lane; e < p.d; e += 32) dst[e] = src[e];
      continue;
    }
    const T *wt = (const T *)(h < p.Hq ? p.qw : p.kw);
    float ss = 0.f;
    for (int e = lane; e < p.d; e += 32) {
      const float x = to_f32(src[e]);
      row[e] = x;
      ss = fmaf(x, x, ss);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = wt ? rsqrtf(fmaf(ss, p.inv_d, p.eps)) : 1.f;
    __syncwarp();
    for (int i = lane; i < p.half; i += 32) {
      const int eu = p.interleaved ? 2 * i : i, ev = p.interleaved ? 2 * i + 1 : i + p.half;
      float sn, cs;
      angle(p, tok, i, &sn, &cs);
      const float u = row[eu] * (wt ? to_f32(wt[eu]) : 1.f);
      const float v = row[ev] * (wt ? to_f32(wt[ev]) : 1.f);
      dst[eu] = from_f32<T>((u * cs - v * sn) * r);
      dst[ev] = from_f32<T>((v * cs + u * sn) * r);
    }
    for (int e = 2 * p.half + lane; e < p.d; e += 32)
      dst[e] = from_f32<T>(row[e] * (wt ? to_f32(wt[e]) : 1.f) * r);
    __syncwarp();
  }
}

}  // namespace nr
}  // namespace gqa
