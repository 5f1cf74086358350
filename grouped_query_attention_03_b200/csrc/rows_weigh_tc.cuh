// rows_weigh_tc.cuh -- what each cell received, from the keys: the second
// kernel of gqa_decode_scored (bf16, d = 64 or 128) for many rows.
//
//   weights[b,g,j] += sum over the lane's R rows rho, j <= its cell, of
//                     2^(s_rho,j - m_rho) / l_rho,   s = scale log2(e) q . k
// with the rows' m and 1 / l from the attention that ran before.  Reading
// the keys again (2 d bytes a cell, from DRAM: the attention lets them go from
// L2 first) and multiplying them again costs less than writing and reading R
// scores of 4 bytes from R = d / 4 rows on.
//
// The product is taken transposed, S^T = K Q^T: a key per TMEM lane, so its
// sum over the rows stays in one thread, without shuffles or atomics, and
// every cell belongs to one CTA.  A CTA has a range of (lane, key tile)
// pairs; a lane's rows are taken 128 at a time, all tiles of its run for
// each:
//   warp 0     TMA producer: Q tiles (2 buffers), K tiles (ring)
//   warp 1     tcgen05.mma S^T (M = 128 keys, N = 128 rows, K = d), four
//              buffers of TMEM
//   warps 4-11 exponentials and sums; the two warpgroups take the tiles in
//              turn and never wait for each other within a run
// Bound by the exponentials: 128 x 128 of them per tile and 128 rows (8 lanes of
// 32768 cells, 128 rows of 128: 20 us, of which the exponentials need 7 and the
// keys' 67 MB 10).
#pragma once

#include "rows_splitk.cuh"

namespace gqa {
namespace rows {

template <int D>
struct WgCfg {
  static constexpr int KB = D / 64;
  static constexpr int BLK = 128 * 128;
  static constexpr int TILE = KB * BLK;
  static constexpr int STAGES = 4;
  static constexpr int OFF_K = 2 * TILE;
  static constexpr int BYTES = OFF_K + STAGES * TILE;
  // at least 120 KB, so that only one CTA (which holds all 512 TMEM columns)
  // is resident per SM
  static constexpr int SMEM = (BYTES + 1024 > 120 * 1024 ? BYTES + 1024 : 120 * 1024);
};

struct WgShared {
  uint64_t q_full[2], q_empty[2], k_full[4], k_empty[4], s_full[4], s_empty[4], mma_fin;
  uint32_t tmem;
  int b, g, tile;
  long long start, end;
  int32_t len[kLenCache];
  // read four at a time
  alignas(16) float m[2][kM];    // [run & 1]: the 128 rows' -m and 1 / l
  alignas(16) float inv[2][kM];
};

// Walks the CTA's range: runs of one lane's tiles.  (Lengths below t hold no
// rows: length_ok keeps them out.)
struct WgWalk {
  int b, g, tile;
  long long pos, end;
  const int32_t *cached;
  __device__ __forceinline__ bool next(const Params &p, int *rb, int *rg, int *rn, int *j0, int *j1) {
    while (true) {
      if (pos >= end || b >= p.B) return false;
      const int n = b < kLenCache ? cached[b] : p.seq_lens[b];
      const int nt = tiles_of(p, n);
      if (nt == 0) {
        ++b;
        g = 0;
        continue;
      }
      *rb = b;
      *rg = g;
      *rn = n;
      *j0 = tile;
      *j1 = (int)min((long long)nt, tile + (end - pos));
      pos += *j1 - *j0;
      tile = 0;
      if (++g == p.Hkv) {
        g = 0;
        ++b;
      }
      return true;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    rows_weigh_tc_kernel(const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK, const Params p) {
  using K = WgCfg<D>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ WgShared sh;
  unsigned char *smem = reinterpret_cast<unsigned char *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sh.s_full[s], 1);
      mbar_init(&sh.s_empty[s], 4);  // the warpgroup that reads S
    }
    for (int s = 0; s < K::STAGES; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 1);
    }
    mbar_init(&sh.mma_fin, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(&sh.tmem, 512);
    tc::tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tmQ);
    tc::prefetch_tmap(&tmK);
  }
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  if (warp == 0) {
    // an even split of all (lane, key tile) pairs
    long long tot = 0;
    for (int b = lane; b < p.B; b += 32) {
      const int n = p.seq_lens[b];
      if (b < kLenCache) sh.len[b] = n;
      tot += tiles_of(p, n);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
    __syncwarp();
    const long long total = tot * p.Hkv, per = (total + gridDim.x - 1) / gridDim.x;
    const long long start = (long long)blockIdx.x * per, end = min(total, start + per);
    long long cum = 0;
    int b = 0, g = 0, tile = 0;
    for (int b0 = 0; b0 < p.B && start < end; b0 += 32) {
      const int bb = b0 + lane;
      const long long x =
          bb < p.B ? (long long)tiles_of(p, bb < kLenCache ? sh.len[bb] : p.seq_lens[bb]) * p.Hkv : 0;
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
        const int nt = (int)(__shfl_sync(0xffffffffu, x, src) / p.Hkv);
        g = (int)((start - cum) / nt);
        tile = (int)((start - cum) - (long long)g * nt);
        break;
      }
      cum += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      sh.b = b;
      sh.g = g;
      sh.tile = tile;
      sh.start = start;
      sh.end = end;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  bool failed = false;
  WgWalk walk{sh.b, sh.g, sh.tile, sh.start, sh.end, sh.len};
  const int MQ = (p.R + kM - 1) / kM;  // 128-row groups of a lane
  int b, g, n, j0, j1;

  if (warp >= 4) {
    const int wg = (warp - 4) >> 2, q4 = warp & 3;
    const int key = q4 * 32 + lane;  // within the tile
    const uint32_t tS0 = tmem + ((uint32_t)(q4 * 32) << 16);
    const float sc = p.scale_log2 == 0.f ? 1e-30f : p.scale_log2;
    const float masked = sc < 0.f ? INFINITY : -INFINITY;  // 2^(sc masked) = 0
    int step = 0, run = 0;
    bool ok = true;
    // (a warp whose wait ran out skips its work but walks on through every
    // run's barrier, which its fellows wait at without a limit)
    while (walk.next(p, &b, &g, &n, &j0, &j1)) {
      const long long ln = (long long)b * p.Hkv + g;
      float *w = p.weights + ln * p.C;
      for (int q = 0; q < MQ; ++q, ++run) {
        const int rb = run & 1;
        // the rows' statistics (rows past the lane's: weight 0).  Written by
        // the first warpgroup; the buffer's last readers have passed the
        // barrier of the run between.
        if (wg == 0) {
          const int rho = q * kM + key;
          const float2 y = rho < p.R ? p.lse[ln * p.R + rho] : make_float2(0.f, 0.f);
          sh.m[rb][key] = -y.x;
          sh.inv[rb][key] = y.y;
        }
        any_of_softmax(false, 256);
        const int step_end = step + (j1 - j0);
        for (int j = j0; ok && j < j1; ++j, ++step) {
          if ((step & 1) != wg) continue;
          const int sb = step & 3;
          const int cell = j * kTile + key;
          const float old = cell < n ? w[cell] : 0.f;  // one thread per run; a barrier between runs
          if (!__all_sync(0xffffffffu, mbar_wait(&sh.s_full[sb], (step >> 2) & 1, &failed))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const bool edge = (j + 1) * kTile > n - p.t + 1;  // some row may not read all of it
          const int behind = cell - (n - p.t);              // row i reads the cell if i >= behind
          const float2 sc2 = make_float2(sc, sc);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          int i = (q * kM) % p.t;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float s[64];
            tc::tmem_ld32(tS0 + sb * kTile + half * 64, s);
            tc::tmem_ld32(tS0 + sb * kTile + half * 64 + 32, s + 32);
            tc::tmem_wait_ld();
            if (half == 1) {
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh.s_empty[sb]);
            }
            const float4 *m4 = reinterpret_cast<const float4 *>(&sh.m[rb][half * 64]);
            const float4 *i4 = reinterpret_cast<const float4 *>(&sh.inv[rb][half * 64]);
            if (edge) {
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                if (i < behind) s[e] = masked;
                if (++i == p.t) i = 0;
              }
            }
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const float4 m = m4[e / 4], inv = i4[e / 4];
              const float2 x = ffma2v(make_float2(s[e], s[e + 1]), sc2, make_float2(m.x, m.y));
              const float2 y = ffma2v(make_float2(s[e + 2], s[e + 3]), sc2, make_float2(m.z, m.w));
              sum[0] = ffma2v(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(inv.x, inv.y), sum[0]);
              sum[1] = ffma2v(make_float2(ex2_approx(y.x), ex2_approx(y.y)), make_float2(inv.z, inv.w), sum[1]);
            }
          }
          if (cell < n) w[cell] = old + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        }
        step = step_end;
      }
    }
  } else if (warp == 0) {
    if (lane == 0) {
      int nq = 0, nk = 0;
      bool ok = true;
      while (ok && walk.next(p, &b, &g, &n, &j0, &j1)) {
        const int ln = b * p.Hkv + g;
        for (int q = 0; ok && q < MQ; ++q) {
          const int qs = nq & 1;
          if (nq >= 2 && !mbar_wait(&sh.q_empty[qs], ((nq >> 1) - 1) & 1, &failed)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sh.q_full[qs], K::TILE);
#pragma unroll
          for (int c = 0; c < K::KB; ++c)
            tc::tma_load_3d(smem + qs * K::TILE + c * K::BLK, &tmQ, c * 64, q * kM, ln, &sh.q_full[qs]);
          ++nq;
          for (int j = j0; j < j1; ++j) {
            const int st = nk % K::STAGES;
            if (nk >= K::STAGES && !mbar_wait(&sh.k_empty[st], (nk / K::STAGES - 1) & 1, &failed)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sh.k_full[st], K::TILE);
#pragma unroll
            for (int c = 0; c < K::KB; ++c)
              tc::tma_load_3d(smem + K::OFF_K + st * K::TILE + c * K::BLK, &tmK, c * 64, j * kTile, ln,
                              &sh.k_full[st]);
            ++nk;
          }
        }
      }
      // Never leave a copy in flight into an exiting CTA: each that was asked
      // for is waited for, whatever became of the others.
      auto landed = [&](uint64_t *bar, int parity) {
        bool late = false;
        mbar_wait(bar, parity, &late);
        failed |= late;
      };
      for (int k = max(0, nq - 2); k < nq; ++k) landed(&sh.q_full[k & 1], (k >> 1) & 1);
      for (int k = max(0, nk - K::STAGES); k < nk; ++k)
        landed(&sh.k_full[k % K::STAGES], (k / K::STAGES) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idS = tc::idesc_bf16_f32(kTile, kM, 0, 0);
      int nq = 0, step = 0;
      bool ok = true;
      while (ok && walk.next(p, &b, &g, &n, &j0, &j1)) {
        for (int q = 0; ok && q < MQ; ++q, ++nq) {
          const uint32_t sQ = smem_u32(smem + (nq & 1) * K::TILE);
          if (!mbar_wait(&sh.q_full[nq & 1], (nq >> 1) & 1, &failed)) {
            ok = false;
            break;
          }
          for (int j = j0; j < j1; ++j, ++step) {
            const int st = step % K::STAGES, sb = step & 3;
            if (!mbar_wait(&sh.k_full[st], (step / K::STAGES) & 1, &failed) ||
                (step >= 4 && !mbar_wait(&sh.s_empty[sb], ((step >> 2) - 1) & 1, &failed))) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const uint32_t sK = smem_u32(smem + K::OFF_K + st * K::TILE);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * K::BLK + (kk & 3) * 32;
              tc::mma_bf16_ss(tmem + sb * kTile, tc::sw128_desc(sK + off, 16, 1024),
                              tc::sw128_desc(sQ + off, 16, 1024), idS, kk > 0 ? 1u : 0u);
            }
            tc::mma_commit(&sh.s_full[sb]);
            tc::mma_commit(&sh.k_empty[st]);
          }
          tc::mma_commit(&sh.q_empty[nq & 1]);
        }
      }
      tc::mma_commit(&sh.mma_fin);
      bool f2 = false;
      mbar_wait(&sh.mma_fin, 0, &f2);
      failed |= f2;
    }
  }
  if (failed) record_status(p.status, kStatusTimeout);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

}  // namespace rows
}  // namespace gqa
