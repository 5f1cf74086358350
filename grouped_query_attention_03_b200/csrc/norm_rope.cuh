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
// F = frac(inv_freq / 2 pi) as a 64-bit fixed-point fraction; position * F in
// wrapping 64-bit integers IS the fraction of the angle, with |position| times
// F's error.  The quotient is therefore formed in two parts (the rounded fp64
// product with 1 / 2 pi, and its remainder with the next 53 bits of it): for
// |inv_freq| up to 2^40 F is within 2^-63.9 turns, the angle of any 32-bit
// position within 2^-32.9.  Its top 32 bits go to sincospif as a signed half
// turn in [-1, 1), rounded to fp32 there (2^-25 half turns).
//
// Each element is read and written once; what stands between that and the
// memory's rate is instructions, about 60 for the 16 bytes a lane has of a
// row.  vec kernel: a group of G = 8, 16 or 32 lanes owns a token, the CTA's
// groups consecutive tokens (a head's output rows are written as one run)
// and a range of heads, all of them where there are tokens enough.  The
// CTA first puts its tokens' cosines and sines in shared memory, each
// computed once; a lane multiplies its own into the weights once for all
// query heads and once for all key heads, so a row costs a sum of squares,
// the exchange of the other half of each pair (shuffles) and two packed FMAs
// per pair of elements.  generic kernel: any width and alignment, a warp per
// row through shared memory.
#pragma once

#include "common.cuh"

namespace gqa {
namespace nr {

constexpr int kMaxAxes = 4;
constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // rows a group has in flight

struct Params {
  const void *qkv, *qw, *kw;
  const float *inv_freq;
  const int32_t *positions;  // [axes,B,T] or NULL (position t)
  void *q, *k, *v;
  int64_t batch_stride, row_stride;  // elements
  int64_t tokens;                    // B * T
  int Hq, Hkv, T, d, half, interleaved;
  int hpg;  // heads per CTA
  float eps, inv_d;
  uint32_t axis[8];  // pair i's axis in bits 2 (i % 16) of word i / 16
};

// frac(f / 2 pi) * 2^64, modulo 2^64.  t - rint(t) is exact; with |f| <= 2^40
// the rest is below 2^-14 and its own rounding below 2^-67.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  constexpr double kInv2Pi = 0.15915494309189535, kInv2PiLow = -9.839338337591243e-18;
  constexpr double kTurn = 18446744073709551616.0;
  const double t = (double)f * kInv2Pi;
  const double rest = fma((double)f, kInv2PiLow, fma((double)f, kInv2Pi, -t));
  return (uint64_t)__double2ll_rn((t - rint(t)) * kTurn) + (uint64_t)__double2ll_rn(rest * kTurn);
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

// A 16-byte vector as fp32 pairs.
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float2 *x) {
    x[0] = make_float2(bf16lo_to_f32(u.x), bf16hi_to_f32(u.x));
    x[1] = make_float2(bf16lo_to_f32(u.y), bf16hi_to_f32(u.y));
    x[2] = make_float2(bf16lo_to_f32(u.z), bf16hi_to_f32(u.z));
    x[3] = make_float2(bf16lo_to_f32(u.w), bf16hi_to_f32(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2 *x) {
    return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y),
                      pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 u, float2 *x) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2 *x) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  }
};

__device__ __forceinline__ float2 fmul2v(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
  return *reinterpret_cast<float2 *>(&d);
}

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
// are the same places of one other lane's vector.  INTER: the (2i, 2i + 1)
// pairing.  PART: some elements are not rotated.
// Five CTAs per SM (48 registers: the compiler spills 40 to 60 bytes a thread in
// bf16, 8 in fp32) and streaming stores: 138 us for 32768 tokens of 48 heads of
// 128 (805 MB moved, 0.89 of the copy rate), against 142 with four and plain
// stores; more rows in flight per group, or the next ones fetched ahead,
// cost registers and gain nothing (138-148).
template <typename T, int G, bool INTER, bool PART>
__global__ void __launch_bounds__(kThreads, 5) norm_rope_vec_kernel(const Params p) {
  constexpr int N = Vec<T>::N, H = N / 2, U = kUnroll;
  constexpr int TOK = kThreads / G;                // tokens per CTA
  constexpr int MAXHALF = G * N / 2;
  __shared__ __align__(16) float s_cos[TOK][MAXHALF], s_sin[TOK][MAXHALF];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int gl = threadIdx.x % G, grp = threadIdx.x / G;
  const int64_t tok0 = (int64_t)blockIdx.x * TOK, tok = tok0 + grp;
  const bool mine = tok < p.tokens;
  const int64_t b = mine ? tok / p.T : 0, t = mine ? tok - b * p.T : 0;
  const int e0 = gl * N;  // first element of this lane
  const bool on = mine && e0 < p.d;
  const int hn = p.Hq + p.Hkv;
  const int h_first = blockIdx.y * p.hpg, h_last = min(h_first + p.hpg, hn + p.Hkv);
  const T *src = (const T *)p.qkv + b * p.batch_stride + t * p.row_stride + e0;
  const unsigned full = 0xffffffffu;

  uint4 raw[U];
  auto load = [&](int h, int end) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      raw[u] = (on && h + u < end) ? ld_stream(src + (int64_t)(h + u) * p.d) : make_uint4(0, 0, 0, 0);
  };
  load(h_first, min(h_last, h_first < p.Hq ? p.Hq : hn));

  if (h_first < hn && p.half > 0) {
    for (int i = threadIdx.x; i < TOK * p.half; i += kThreads) {
      const int k = i / p.half, pair = i - k * p.half;
      if (tok0 + k < p.tokens) angle(p, tok0 + k, pair, &s_sin[k][pair], &s_cos[k][pair]);
    }
  }
  __syncthreads();

  // where this lane's partners are
  const int hv = p.half / N;  // lanes from one half to the other
  const bool lowhalf = gl < hv;
  const int partner = (INTER || gl >= 2 * hv) ? gl : (lowhalf ? gl + hv : gl - hv);
  // y = r (x A + x_partner B),  A = w cos, B = +-w_partner sin, r = 1 / sqrt(
  // mean + eps).  Past rot there is no partner (and inf * 0 is not 0).
  float2 A[H], B[H];
  bool turned[H];
  auto weigh = [&](const T *w) {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int e = e0 + 2 * i;
      turned[i] = on && e < 2 * p.half;
      float2 w2 = make_float2(1.f, 1.f), wp = w2;
      if (w && on) {
        w2 = make_float2(to_f32(w[e]), to_f32(w[e + 1]));
        const int pe = partner * N + 2 * i;
        wp = INTER ? make_float2(w2.y, w2.x) : make_float2(to_f32(w[pe]), to_f32(w[pe + 1]));
      }
      A[i] = w2;
      B[i] = make_float2(0.f, 0.f);
      if (turned[i]) {
        if (INTER) {
          const float c = s_cos[grp][e / 2], n = s_sin[grp][e / 2];
          A[i] = make_float2(w2.x * c, w2.y * c);
          B[i] = make_float2(-wp.x * n, wp.y * n);
        } else {
          const int pair = lowhalf ? e : e - p.half;
          const float sg = lowhalf ? -1.f : 1.f;
          A[i] = make_float2(w2.x * s_cos[grp][pair], w2.y * s_cos[grp][pair + 1]);
          B[i] = make_float2(sg * wp.x * s_sin[grp][pair], sg * wp.y * s_sin[grp][pair + 1]);
        }
      }
    }
  };

  // heads [h, end) of one kind; dst: head h's row of this token
  auto turn_rows = [&](int h, int end, T *dst, bool norm) {
    const int64_t step = (int64_t)p.T * p.d;
    for (; h < end; h += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (h + u >= end) break;  // the same for all lanes
        float2 x[H], xp[H], ss2 = make_float2(0.f, 0.f);
        Vec<T>::unpack(raw[u], x);
        float r = 1.f;
        if (norm) {
#pragma unroll
          for (int i = 0; i < H; ++i) ss2 = ffma2v(x[i], x[i], ss2);
          float ss = ss2.x + ss2.y;
#pragma unroll
          for (int off = G / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(full, ss, off);
          r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
        }
        if (INTER) {
#pragma unroll
          for (int i = 0; i < H; ++i) xp[i] = make_float2(x[i].y, x[i].x);
        } else {
          uint4 o;
          o.x = __shfl_sync(full, raw[u].x, partner, G);
          o.y = __shfl_sync(full, raw[u].y, partner, G);
          o.z = __shfl_sync(full, raw[u].z, partner, G);
          o.w = __shfl_sync(full, raw[u].w, partner, G);
          Vec<T>::unpack(o, xp);
        }
        const float2 r2 = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          float2 y = fmul2v(x[i], A[i]);
          if (!PART || turned[i]) y = ffma2v(xp[i], B[i], y);
          x[i] = fmul2v(y, r2);
        }
        if (on) __stcs(reinterpret_cast<uint4 *>(dst + u * step), Vec<T>::pack(x));
      }
      dst += U * step;
      load(h + U, end);
    }
  };
  auto row_of = [&](void *out, int heads, int h) {
    return (T *)out + ((b * heads + h) * p.T + t) * p.d + e0;
  };
  int h = h_first;
  if (h < p.Hq) {
    const int end = min(h_last, p.Hq);
    weigh((const T *)p.qw);
    turn_rows(h, end, row_of(p.q, p.Hq, h), p.qw != nullptr);
    h = end;
    load(h, min(h_last, hn));
  }
  if (h < h_last && h < hn) {
    const int end = min(h_last, hn);
    weigh((const T *)p.kw);
    turn_rows(h, end, row_of(p.k, p.Hkv, h - p.Hq), p.kw != nullptr);
    h = end;
  }
  if (h < h_last) {  // values: as they are
    const int64_t step = (int64_t)p.T * p.d;
    T *dst = row_of(p.v, p.Hkv, h - hn);
    for (; h < h_last; h += U, dst += U * step) {
      load(h, h_last);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (on && h + u < h_last) __stcs(reinterpret_cast<uint4 *>(dst + u * step), raw[u]);
    }
  }
}

// Any width up to GQA_MAX_HEAD_DIM, any alignment: a warp per row, which works
// its token's angles out itself (bf16, 48 heads of 80, halves of 38, 4096 tokens:
// 110 us of 10 at the copy rate; fp32, 12 heads of 256, 2000 tokens: 20 of 7.5).
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
