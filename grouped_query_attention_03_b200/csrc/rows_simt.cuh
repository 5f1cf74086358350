// rows_simt.cuh -- CUDA-core kernel of gqa_decode_tree and
// gqa_decode_scored: fp32 tensors (fp32 FMAs, see simt.cuh) and the bf16
// head widths that the tensor-core kernel is not compiled for.
//
// CTA = (part, group of 16 rows, lane): the lane's keys (cells, then drafts)
// are cut into ns equal parts.  32 keys at a time pass through shared
// memory as fp32: each thread scores one key against 4 rows (the key's
// features in its registers' reach, the rows' broadcast), the 4 warps run
// the online softmax of 4 rows each, lane = key, and each thread mixes the
// values of up to 2 columns for all 16 rows.  Bound by shared-memory reads:
// 5 per 16 FMAs in both products.
#pragma once

#include "rows.cuh"

namespace gqa {
namespace rows {

constexpr int kSR = 16;  // rows per CTA
constexpr int kSK = 32;  // keys per step
constexpr int kSimtThreads = 128;

__host__ __device__ constexpr int simt_pitch(int d) { return ((d + 3) / 4) * 4 + 4; }
inline int simt_smem(int d) { return (kSR + kSK) * simt_pitch(d) * 4 + kSK * kSR * 4; }

template <typename T>
__global__ void __launch_bounds__(kSimtThreads) rows_simt_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int32_t s_par[kMaxNodes];
  __shared__ float s_alpha[kSR], s_ml[kSR][2];
  __shared__ int s_last;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int pitch = simt_pitch(p.d), d4 = (p.d + 3) / 4;
  float *sq = sm, *skv = sq + kSR * pitch, *sp = skv + kSK * pitch;  // sp [key][row]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // blockIdx.x = (lane (b, g) * MG + group) * ns + part
  const long long L = (long long)blockIdx.x / p.ns;  // lane group
  const int part = (int)(blockIdx.x - L * p.ns);
  const int grp = (int)(L % p.MG);
  const long long ln = L / p.MG;
  const int b = (int)(ln / p.Hkv), g = (int)(ln - (long long)b * p.Hkv);
  const int rho0 = grp * kSR, nrows = min(kSR, p.R - rho0);
  const long long row0 = ((long long)b * p.Hq + (long long)g * p.r) * p.t + rho0;
  const int n = p.seq_lens[b];
  T *o = (T *)p.o + row0 * p.d;
  const long long slot = L * p.ns + part;
  if (!length_ok(p, n)) {
    if (tid == 0) record_status(p.status, GQA_ERR_CAPACITY);
    if (part == 0)
      for (int i = tid; i < nrows * p.d; i += kSimtThreads) o[i] = from_f32<T>(0.f);
    return;
  }
  if (p.tree && p.parents)
    for (int i = tid; i < p.t; i += kSimtThreads) s_par[i] = p.parents[(long long)b * p.t + i];
  for (int i = tid; i < kSR * pitch; i += kSimtThreads) {
    const int row = i / pitch, c = i - row * pitch;
    sq[i] = (row < nrows && c < p.d) ? to_f32(((const T *)p.q)[(row0 + row) * p.d + c]) * p.scale_log2
                                     : 0.f;
  }
  __syncthreads();
  // this warp's 4 rows: what they may read
  const int lo0 = first_cell(p, n), nc = n - lo0;
  const int nkeys = nc + (p.tree ? p.t : 0);
  int lo[4], hi[4];  // cells [lo, hi) of each row
  Line line[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = warp * 4 + k, i = (rho0 + row) % p.t;
    lo[k] = 0;
    hi[k] = 0;
    line[k].depth = -1;
#pragma unroll
    for (int w = 0; w < kMaxNodes / 32; ++w) line[k].bits[w] = 0u;
    if (row >= nrows) continue;
    if (p.tree) {
      line[k] = line_of(p.parents ? s_par : nullptr, i, p.window);
      if (line[k].refused && lane == 0) record_status(p.status, GQA_ERR_TREE);
      if (line[k].depth >= 0) {
        lo[k] = p.window > 0 ? max(0, n + line[k].depth - (p.window - 1)) : 0;
        hi[k] = n;
      }
    } else {
      hi[k] = n - p.t + i + 1;
    }
  }
  // keys [k0, k1) of the lane
  const int k0 = (int)((long long)nkeys * part / p.ns);
  const int k1 = (int)((long long)nkeys * (part + 1) / p.ns);
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, l[4] = {0.f, 0.f, 0.f, 0.f};
  float acc[2][kSR];
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int k = 0; k < kSR; ++k) acc[c][k] = 0.f;

  // K (or V) rows of keys [kb, kb + 32) to shared memory; true if a value is
  // not finite
  auto stage = [&](const void *cache, const void *draft, int kb) -> bool {
    bool odd = false;
    for (int i = tid; i < kSK * pitch; i += kSimtThreads) {
      const int key = i / pitch, c = i - key * pitch, kk = kb + key;
      float x = 0.f;
      if (kk < k1 && c < p.d) {
        if (kk < nc)
          x = to_f32(((const T *)cache)[(ln * p.C + lo0 + kk) * p.d + c]);
        else
          x = to_f32(((const T *)draft)[(ln * p.t + (kk - nc)) * p.d + c]);
      }
      odd |= !isfinite(x);
      skv[i] = x;
    }
    return odd;
  };

  for (int kb = k0; kb < k1; kb += kSK) {
    __syncthreads();  // the last step's values and weights are used up
    stage(p.k, p.kd, kb);
    __syncthreads();
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const float4 *k4 = reinterpret_cast<const float4 *>(skv + lane * pitch);
    const float4 *q4 = reinterpret_cast<const float4 *>(sq + warp * 4 * pitch);
    const int p4 = pitch / 4;
    for (int c = 0; c < d4; ++c) {
      const float4 kv = k4[c];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 qv = q4[k * p4 + c];
        s[k] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[k]))));
      }
    }
    const int kk = kb + lane, cell = lo0 + kk, node = kk - nc;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      bool ok = kk < k1;
      if (kk < nc) {
        ok = ok && cell >= lo[k] && cell < hi[k];
      } else {
        uint32_t word = 0u;
#pragma unroll
        for (int w = 0; w < kMaxNodes / 32; ++w)
          if ((node >> 5) == w) word = line[k].bits[w];
        ok = ok && ((word >> (node & 31)) & 1u);
      }
      if (!ok) s[k] = -INFINITY;
      const int rho = rho0 + warp * 4 + k;
      if (p.scores && kk < k1 && warp * 4 + k < nrows)
        p.scores[(ln * p.R + rho) * p.Cp + cell] = s[k];
      float mx = s[k];
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float m_new = fmaxf(m[k], mx);
      const float msub = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m[k] - msub);  // 0 from -inf
      const float pv = exp2f(s[k] - msub);
      float ps = pv;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
      l[k] = fmaf(l[k], alpha, ps);
      m[k] = m_new;
      sp[lane * kSR + warp * 4 + k] = pv;
      if (lane == 0) s_alpha[warp * 4 + k] = alpha;
    }
    __syncthreads();  // scores taken from skv; sp, s_alpha complete
    // a value that is not finite must not reach rows that may not read it
    const bool odd = __syncthreads_or(stage(p.v, p.vd, kb)) != 0;
    float al[kSR];
#pragma unroll
    for (int k = 0; k < kSR; ++k) al[k] = s_alpha[k];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = tid + c * kSimtThreads;
      if (col >= p.d) continue;
#pragma unroll
      for (int k = 0; k < kSR; ++k) acc[c][k] *= al[k];
      for (int key = 0; key < kSK; ++key) {
        const float v = skv[key * pitch + col];
        const float4 *w4 = reinterpret_cast<const float4 *>(sp + key * kSR);
        float w[kSR];
#pragma unroll
        for (int k = 0; k < kSR / 4; ++k) {
          const float4 y = w4[k];
          w[4 * k] = y.x; w[4 * k + 1] = y.y; w[4 * k + 2] = y.z; w[4 * k + 3] = y.w;
        }
        if (odd) {
#pragma unroll
          for (int k = 0; k < kSR; ++k)
            if (w[k] != 0.f) acc[c][k] = fmaf(w[k], v, acc[c][k]);
        } else {
#pragma unroll
          for (int k = 0; k < kSR; ++k) acc[c][k] = fmaf(w[k], v, acc[c][k]);
        }
      }
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s_ml[warp * 4 + k][0] = m[k];
      s_ml[warp * 4 + k][1] = l[k];
    }
  }
  __syncthreads();
  if (p.ns == 1) {
    if (p.lse && tid < nrows) {
      const float mk = s_ml[tid][0], lk = s_ml[tid][1];
      p.lse[ln * p.R + rho0 + tid] =
          make_float2(mk == -INFINITY ? 0.f : mk, lk == 0.f ? 0.f : 1.f / lk);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = tid + c * kSimtThreads;
      if (col >= p.d) continue;
#pragma unroll
      for (int k = 0; k < kSR; ++k) {
        if (k >= nrows) continue;
        const float lk = s_ml[k][1];
        o[(long long)k * p.d + col] = from_f32<T>(lk == 0.f ? 0.f : acc[c][k] / lk);  // 0: no keys
      }
    }
    return;
  }
  if (tid < nrows) p.ml[slot * kSR + tid] = make_float2(s_ml[tid][0], s_ml[tid][1]);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int col = tid + c * kSimtThreads;
    if (col >= p.d) continue;
#pragma unroll
    for (int k = 0; k < kSR; ++k)
      if (k < nrows) p.acc[((slot * d4 + col / 4) * kSR + k) * 4 + (col & 3)] = acc[c][k];
  }
  __syncthreads();
  if (tid == 0) s_last = count_part(&p.counters[L], p.ns);
  __syncthreads();
  if (!s_last) return;
  merge_parts<kSimtThreads / 32>(p, L * p.ns, p.ns, nrows, warp, sm, pitch,
                                 p.lse ? p.lse + ln * p.R + rho0 : nullptr);
  __syncthreads();
  for (int k = warp; k < nrows; k += kSimtThreads / 32)
    for (int c = lane; c < p.d; c += 32) o[(long long)k * p.d + c] = from_f32<T>(sm[k * pitch + c]);
}

}  // namespace rows
}  // namespace gqa
