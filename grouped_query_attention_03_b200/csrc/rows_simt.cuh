// rows_simt.cuh -- CUDA-core kernel of gqa_decode_tree and
// gqa_decode_scored: fp32 tensors (fp32 FMAs, see simt.cuh) and the bf16
// head widths that the tensor-core kernel is not compiled for.
//
// CTA = (part, group of 16 rows, lane): the lane's keys (cells, then drafts)
// are cut into ns equal parts, taken 32 at a time.  A warp scores 4 rows, lane =
// key (the key's features from its row in shared memory, the rows' broadcast),
// and runs their online softmax; then a thread mixes 4 columns of RPT rows.
// With 8 rows or fewer the warps share a row group's features, and the threads
// without rows of their own take a share of the keys in the mix.  Rows of
// whole 16-byte vectors arrive by asynchronous copies: the next keys travel
// under the mix, the values under the scores.
// Bound by shared-memory reads (8 cycles of them per 4 of FMAs in the scores, 5
// in the mix) with many rows, by the latency of a step, about 1.5 us, with few.
// fp32: 4 sequences of 2000 cells, 32 heads of 128 on 8, 32 nodes: 240 us, 18
// TFLOP/s; one head, 58 cells, 2 nodes: 8.8 us.  Four CTAs per SM (128
// registers, of which the compiler spills 12 to 88 bytes a thread) instead of
// as many as unlimited registers leave: 240 us against 308 there, 8.8 against
// 8.6 here.
#pragma once

#include "rows.cuh"

namespace gqa {
namespace rows {

constexpr int kSR = 16;  // rows per CTA
constexpr int kSK = 32;  // keys per step
constexpr int kSimtThreads = 128;
constexpr int kSimtWarps = kSimtThreads / 32;

// Row pitches: queries (floats) and keys or values (bytes).  4 words past a
// multiple of 16 bytes keep a warp's rows in different banks.
__host__ __device__ constexpr int simt_pitch(int d) { return ((d + 3) / 4) * 4 + 4; }
__host__ __device__ constexpr int simt_kv_pitch(int d, int elem) {
  return ((d + 3) / 4 * 4 * elem + 15) / 16 * 16 + 16;
}
inline int simt_smem(int d, int elem) {
  return kSR * simt_pitch(d) * 4 + 2 * kSK * simt_kv_pitch(d, elem) + kSK * kSR * 4;
}

// Rows per thread in the mix: a thread per 4 columns and RPT rows.
inline int simt_rpt(int d) { return d <= 32 ? 1 : d <= 64 ? 2 : d <= 128 ? 4 : 8; }

// 4 elements of a row in shared memory.
template <typename T>
__device__ __forceinline__ float4 row4(const unsigned char *row, int c);
template <>
__device__ __forceinline__ float4 row4<float>(const unsigned char *row, int c) {
  return *reinterpret_cast<const float4 *>(row + c * 16);
}
template <>
__device__ __forceinline__ float4 row4<__nv_bfloat16>(const unsigned char *row, int c) {
  const uint2 u = *reinterpret_cast<const uint2 *>(row + c * 8);
  return make_float4(bf16lo_to_f32(u.x), bf16hi_to_f32(u.x), bf16lo_to_f32(u.y), bf16hi_to_f32(u.y));
}

// 16 bytes to shared memory.
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// RPT weights, at an address of as many floats.
template <int RPT>
__device__ __forceinline__ void load_weights(const float *at, float *w) {
  if constexpr (RPT >= 4) {
#pragma unroll
    for (int k = 0; k < RPT; k += 4) {
      const float4 y = *reinterpret_cast<const float4 *>(at + k);
      w[k] = y.x;
      w[k + 1] = y.y;
      w[k + 2] = y.z;
      w[k + 3] = y.w;
    }
  } else if constexpr (RPT == 2) {
    const float2 y = *reinterpret_cast<const float2 *>(at);
    w[0] = y.x;
    w[1] = y.y;
  } else {
    w[0] = at[0];
  }
}

template <typename T, int RPT>
__global__ void __launch_bounds__(kSimtThreads, 4) rows_simt_kernel(const Params p) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int32_t s_par[kMaxNodes];
  __shared__ __align__(16) float s_alpha[kSR];
  __shared__ float4 s_part[kSimtWarps][kSK];
  __shared__ float s_ml[kSR][2];
  __shared__ int s_last;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int pitch = simt_pitch(p.d), kv_pitch = simt_kv_pitch(p.d, sizeof(T)), d4 = (p.d + 3) / 4;
  float *sq = sm;
  unsigned char *sk = reinterpret_cast<unsigned char *>(sq + kSR * pitch), *sv = sk + kSK * kv_pitch;
  float *sp = reinterpret_cast<float *>(sv + kSK * kv_pitch);  // [key][row]
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
  for (int c = lane; c < pitch; c += 32) {  // (does not wait for the length)
    float x[kSR / kSimtWarps];
#pragma unroll
    for (int u = 0; u < kSR / kSimtWarps; ++u) {
      const int row = warp + u * kSimtWarps;
      x[u] = row < nrows && c < p.d ? to_f32(((const T *)p.q)[(row0 + row) * p.d + c]) * p.scale_log2 : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kSR / kSimtWarps; ++u) sq[(warp + u * kSimtWarps) * pitch + c] = x[u];
  }
  if (!length_ok(p, n)) {
    if (tid == 0) record_status(p.status, GQA_ERR_CAPACITY);
    if (part == 0)
      for (int i = tid; i < nrows * p.d; i += kSimtThreads) o[i] = from_f32<T>(0.f);
    return;
  }
  const int lo0 = first_cell(p, n), nc = n - lo0;
  const int nkeys = nc + (p.tree ? p.t : 0);
  // keys [k0, k1) of the lane
  const int k0 = (int)((long long)nkeys * part / p.ns);
  const int k1 = (int)((long long)nkeys * (part + 1) / p.ns);
  // Rows of keys [kb, min(kb + 32, k1)) to shared memory.  What is behind them
  // stays as it was: its scores are masked and its weights 0.
  // LPK lanes of 16 bytes take a row (d > 128 in fp32: twice)
  constexpr int LPK = RPT * (int)sizeof(T) >= 16 ? 32 : RPT * (int)sizeof(T) >= 8 ? 16 : 8;
  const int v_key = tid / LPK, v_at = tid % LPK * 16, row_bytes = p.d * (int)sizeof(T);
  auto stage = [&](const void *cache, const void *draft, unsigned char *to, int kb) {
    if (p.vec) {
      const char *c0 = (const char *)((const T *)cache + (ln * p.C + lo0) * p.d) + v_at;
      const char *d0 = (const char *)((const T *)draft + ln * p.t * p.d) + v_at;
#pragma unroll
      for (int key = v_key; key < kSK; key += kSimtThreads / LPK) {
        const int kk = kb + key;
        const char *src = kk < nc ? c0 + (long long)kk * row_bytes : d0 + (long long)(kk - nc) * row_bytes;
        unsigned char *dst = to + key * kv_pitch + v_at;
        if (kk < k1) {
          if (v_at < row_bytes) cp_async16(dst, src);
          if (RPT * sizeof(T) == 32 && v_at + LPK * 16 < row_bytes)
            cp_async16(dst + LPK * 16, src + LPK * 16);
        }
      }
    } else {
      constexpr int U = kSK / kSimtWarps;
      for (int c = lane; c < d4 * 4; c += 32) {
        T x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int kk = kb + warp + u * kSimtWarps;
          x[u] = kk >= k1 || c >= p.d ? from_f32<T>(0.f)
                 : kk < nc           ? ((const T *)cache)[(ln * p.C + lo0 + kk) * p.d + c]
                                     : ((const T *)draft)[(ln * p.t + (kk - nc)) * p.d + c];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          reinterpret_cast<T *>(to + (warp + u * kSimtWarps) * kv_pitch)[c] = x[u];
      }
    }
    cp_async_commit();
  };
  if (k0 < k1) {
    stage(p.k, p.kd, sk, k0);
    stage(p.v, p.vd, sv, k0);
  }
  if (p.tree && p.parents)
    for (int i = tid; i < p.t; i += kSimtThreads) s_par[i] = p.parents[(long long)b * p.t + i];
  for (int i = tid; i < kSK * kSR; i += kSimtThreads) sp[i] = 0.f;  // rows past the last stay 0
  if (tid < kSR) {
    s_alpha[tid] = 0.f;
    s_ml[tid][0] = -INFINITY;
    s_ml[tid][1] = 0.f;
  }
  __syncthreads();
  // Warps per 4 rows: they share the rows' features, the first runs the softmax.
  const int wpr = nrows <= 4 ? 4 : nrows <= 8 ? 2 : 1;
  const int r4 = warp / wpr * 4, sub = warp & (wpr - 1);  // this warp's rows, its share
  const int cw = (d4 + wpr - 1) / wpr, c_lo = min(d4, sub * cw), c_hi = min(d4, c_lo + cw);
  const bool scores_on = r4 < nrows, softmax_on = scores_on && sub == 0;
  // what the rows may read; a lane works out row lane % 4
  int lo[4], hi[4];  // cells [lo, hi) of each row
  uint32_t bits[4][kMaxNodes / 32];
  int lo_all = 0, k_all = min(k1, nc);  // keys from cell lo_all to key k_all: all rows
  if (softmax_on) {
    const int row = r4 + (lane & 3), i = (rho0 + row) % p.t;
    Line ln4;
    ln4.depth = -1;
    ln4.refused = false;
#pragma unroll
    for (int w = 0; w < kMaxNodes / 32; ++w) ln4.bits[w] = 0u;
    int lo1 = 0, hi1 = 0;
    if (row < nrows) {
      if (p.tree) {
        ln4 = line_of(p.parents ? s_par : nullptr, i, p.window);
        if (ln4.refused) record_status(p.status, GQA_ERR_TREE);
        if (ln4.depth >= 0) {
          lo1 = p.window > 0 ? max(0, n + ln4.depth - (p.window - 1)) : 0;
          hi1 = n;
        }
      } else {
        hi1 = n - p.t + i + 1;
      }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] = __shfl_sync(0xffffffffu, lo1, k);
      hi[k] = __shfl_sync(0xffffffffu, hi1, k);
#pragma unroll
      for (int w = 0; w < kMaxNodes / 32; ++w) bits[k][w] = __shfl_sync(0xffffffffu, ln4.bits[w], k);
      if (r4 + k < nrows) {
        lo_all = max(lo_all, lo[k]);
        k_all = min(k_all, hi[k] - lo0);
      }
    }
  }
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  float l[4] = {0.f, 0.f, 0.f, 0.f};  // this lane's keys
  // This thread's part of the mix: columns [4 cg, 4 cg + 4) of rows [mr, mr +
  // RPT), keys ks, ks + KS, ...
  constexpr int G = kSR / RPT;  // groups of d4 threads: d4 G <= kSimtThreads
  const int cg = tid % d4, mg = tid / d4;
  int nrg = 1;  // groups of rows
  while (nrg * RPT < nrows) nrg *= 2;
  const int KS = G / nrg, ks = mg / nrg, mr = (mg & (nrg - 1)) * RPT;
  const bool mixes = mg < G && mr < nrows;
  float acc[RPT][4];
#pragma unroll
  for (int k = 0; k < RPT; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;

  for (int kb = k0; kb < k1; kb += kSK) {
    if (kb == k0)
      cp_async_wait<1>();  // the keys (the values were asked for behind them)
    else
      cp_async_wait<0>();
    __syncthreads();  // keys here; the last step's values and weights are used up
    if (kb > k0) stage(p.v, p.vd, sv, kb);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (scores_on) {
      const unsigned char *krow = sk + lane * kv_pitch;
      const float4 *q4 = reinterpret_cast<const float4 *>(sq + r4 * pitch);
      const int p4 = pitch / 4;
#pragma unroll 4
      for (int c = c_lo; c < c_hi; ++c) {
        const float4 kv = row4<T>(krow, c);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 qv = q4[k * p4 + c];
          s[k] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[k]))));
        }
      }
    }
    if (wpr > 1) {
      if (scores_on && sub > 0) s_part[warp][lane] = make_float4(s[0], s[1], s[2], s[3]);
      __syncthreads();
      if (softmax_on)
        for (int u = 1; u < wpr; ++u) {
          const float4 y = s_part[warp + u][lane];
          s[0] += y.x;
          s[1] += y.y;
          s[2] += y.z;
          s[3] += y.w;
        }
    }
    if (softmax_on) {
      const int kk = kb + lane, cell = lo0 + kk, node = kk - nc;
      float mx[4], pv[4], alpha[4];
      if (kb + kSK > k_all || lo0 + kb < lo_all) {  // some row may not read all of these keys
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          bool ok = kk < k1;
          if (kk < nc) {
            ok = ok && cell >= lo[k] && cell < hi[k];
          } else {
            uint32_t word = 0u;
#pragma unroll
            for (int w = 0; w < kMaxNodes / 32; ++w)
              if ((node >> 5) == w) word = bits[k][w];
            ok = ok && ((word >> (node & 31)) & 1u);
          }
          if (!ok) s[k] = -INFINITY;
        }
      }
      if (p.scores && kk < k1) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (r4 + k < nrows) p.scores[(ln * p.R + rho0 + r4 + k) * p.Cp + cell] = s[k];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k] = s[k];
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], off));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float m_new = fmaxf(m[k], mx[k]);
        const float msub = m_new == -INFINITY ? 0.f : m_new;
        alpha[k] = exp2f(m[k] - msub);  // 0 from -inf
        pv[k] = exp2f(s[k] - msub);
        l[k] = fmaf(l[k], alpha[k], pv[k]);
        m[k] = m_new;
      }
      *reinterpret_cast<float4 *>(sp + lane * kSR + r4) = make_float4(pv[0], pv[1], pv[2], pv[3]);
      if (lane == 0)
        *reinterpret_cast<float4 *>(s_alpha + r4) =
            make_float4(alpha[0], alpha[1], alpha[2], alpha[3]);
    }
    cp_async_wait<0>();
    __syncthreads();  // values here; keys used up; sp and s_alpha complete
    if (kb + kSK < k1) stage(p.k, p.kd, sk, kb + kSK);
    if (mixes) {
#pragma unroll
      for (int k = 0; k < RPT; ++k) {
        const float al = s_alpha[mr + k];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[k][j] *= al;
      }
#pragma unroll 4
      for (int key = ks; key < kSK; key += KS) {
        const float4 v = row4<T>(sv + key * kv_pitch, cg);
        float w[RPT];
        load_weights<RPT>(sp + key * kSR + mr, w);
#pragma unroll
        for (int k = 0; k < RPT; ++k)
          // a weight of 0 adds nothing, whatever the value: a row's masked keys
          // may hold what is not finite
          if (w[k] != 0.f) {
            acc[k][0] = fmaf(w[k], v.x, acc[k][0]);
            acc[k][1] = fmaf(w[k], v.y, acc[k][1]);
            acc[k][2] = fmaf(w[k], v.z, acc[k][2]);
            acc[k][3] = fmaf(w[k], v.w, acc[k][3]);
          }
      }
    }
  }
  __syncthreads();  // the queries and the last values are used up
  if (KS > 1) {  // the shares of the keys, through the queries' place, in order
    float *red = sq;
    if (mixes && ks > 0)
#pragma unroll
      for (int k = 0; k < RPT; ++k)
        *reinterpret_cast<float4 *>(red + ((mg * RPT + k) * d4 + cg) * 4) =
            make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
    __syncthreads();
    if (mixes && ks == 0)
      for (int u = 1; u < KS; ++u)
#pragma unroll
        for (int k = 0; k < RPT; ++k) {
          const float4 y =
              *reinterpret_cast<const float4 *>(red + (((u * nrg + mg) * RPT + k) * d4 + cg) * 4);
          acc[k][0] += y.x;
          acc[k][1] += y.y;
          acc[k][2] += y.z;
          acc[k][3] += y.w;
        }
  }
  const bool writes = mixes && ks == 0;
  if (softmax_on) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) l[k] += __shfl_xor_sync(0xffffffffu, l[k], off);
  }
  if (lane == 0 && softmax_on) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s_ml[r4 + k][0] = m[k];
      s_ml[r4 + k][1] = l[k];
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
    for (int k = 0; k < RPT; ++k) {
      if (!writes || mr + k >= nrows) break;
      const float lk = s_ml[mr + k][1], inv = lk == 0.f ? 0.f : 1.f / lk;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (cg * 4 + j < p.d)  // 0: no keys
          o[(long long)(mr + k) * p.d + cg * 4 + j] = from_f32<T>(lk == 0.f ? 0.f : acc[k][j] * inv);
    }
    return;
  }
  if (tid < nrows) p.ml[slot * kSR + tid] = make_float2(s_ml[tid][0], s_ml[tid][1]);
#pragma unroll
  for (int k = 0; k < RPT; ++k)
    if (writes && mr + k < nrows)
      *reinterpret_cast<float4 *>(p.acc + ((slot * d4 + cg) * kSR + mr + k) * 4) =
          make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
  __syncthreads();
  if (tid == 0) s_last = count_part(&p.counters[L], p.ns);
  __syncthreads();
  if (!s_last) return;
  merge_parts<kSimtWarps>(p, L * p.ns, p.ns, nrows, warp, sm, pitch,
                                 p.lse ? p.lse + ln * p.R + rho0 : nullptr);
  __syncthreads();
  for (int k = warp; k < nrows; k += kSimtWarps)
    for (int c = lane; c < p.d; c += 32) o[(long long)k * p.d + c] = from_f32<T>(sm[k * pitch + c]);
}

// ------------------------------------------------------------------ weights
// What each cell received, from the keys: for many scored rows of the bf16
// types that the tensor-core kernel takes (which keeps no scores for them, see
// rows_weigh_tc.cuh), in buffers that are not aligned for it.  The workspace
// query does not know the alignment, so the scores are not kept here either.
// Block = 64 cells of a lane, two threads per cell: its key in shared memory,
// 16 rows' features and statistics at a time, 8 rows' products together in
// each.  Bound by shared-memory reads, like the scores above (8 lanes of 32768
// cells, 128 rows of 128: 1.91 ms with the attention, against 1.63 with 134 MB of
// scores kept; 8 lanes of 2000, 64 rows of 64: 95 us and 69).
constexpr int kWeighKeys = 64, kWeighRows = 16, kWeighKeyThreads = 2 * kWeighKeys;

template <int D>
__global__ void __launch_bounds__(kWeighKeyThreads) rows_weigh_keys_kernel(const Params p, int cell_blocks) {
  constexpr int PITCH = 2 * D + 8;  // bytes: a warp's 8-byte reads meet no bank twice
  __shared__ __align__(16) unsigned char keys[kWeighKeys * PITCH];
  __shared__ __align__(16) float q[kWeighRows][D];
  __shared__ float s_m[kWeighRows], s_inv[kWeighRows], s_w[kWeighKeys];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int tid = threadIdx.x, key = tid % kWeighKeys, k0 = tid / kWeighKeys * 8;
  const long long ln = blockIdx.x / cell_blocks;
  const int j0 = (int)(blockIdx.x - ln * cell_blocks) * kWeighKeys, cell = j0 + key;
  const int b = (int)(ln / p.Hkv), n = p.seq_lens[b];
  if (!length_ok(p, n) || j0 >= n) return;
  const __nv_bfloat16 *k = (const __nv_bfloat16 *)p.k + (ln * p.C + j0) * D;
  for (int i = tid; i < kWeighKeys * D; i += kWeighKeyThreads)
    if (j0 + i / D < n) *reinterpret_cast<__nv_bfloat16 *>(keys + i / D * PITCH + i % D * 2) = k[i];
  float w = 0.f;
  for (int r0 = 0; r0 < p.R; r0 += kWeighRows) {
    const int nr = min(kWeighRows, p.R - r0);
    __syncthreads();
    for (int i = tid; i < kWeighRows * D; i += kWeighKeyThreads)
      q[i / D][i % D] =
          i / D < nr ? to_f32(((const __nv_bfloat16 *)p.q)[(ln * p.R + r0) * D + i]) * p.scale_log2 : 0.f;
    if (tid < nr) {
      const float2 x = p.lse[ln * p.R + r0 + tid];
      s_m[tid] = x.x;
      s_inv[tid] = x.y;
    }
    __syncthreads();
    if (cell >= n || k0 >= nr) continue;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = 0; c < D / 4; ++c) {
      const float4 kv = row4<__nv_bfloat16>(keys + key * PITCH, c);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float4 qv = *reinterpret_cast<const float4 *>(&q[k0 + u][c * 4]);
        s[u] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, s[u]))));
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)  // row i reads the cell if it is at or before its own
      if (k0 + u < nr && cell <= n - p.t + (r0 + k0 + u) % p.t)
        w = fmaf(exp2f(s[u] - s_m[k0 + u]), s_inv[k0 + u], w);
  }
  if (k0 > 0) s_w[key] = w;
  __syncthreads();
  if (k0 == 0 && cell < n) p.weights[ln * p.C + cell] += w + s_w[key];
}

}  // namespace rows
}  // namespace gqa
