// tree_commit.cuh -- the accepted path of a drafted tree enters the cache.
//
// Row path[b][j] of the drafted keys and values goes to cell len_b + j of
// its lane, j < path_len_b, and the length becomes len_b + path_len_b: an
// append of selected rows, all-or-nothing over the batch like the append.
// A handful of rows per sequence, so latency is what counts: one thread per
// 16-byte column of a lane, its rows loaded in batches of 8.
//
// The lengths may be advanced in place.  Every CTA checks every length
// before it writes, so they change only after the last CTA has read them:
//   commit = 1  this launch writes lens_out: another buffer than seq_lens,
//               or one cluster that passes its barrier first
//   commit = 0  tree_commit_lens_kernel follows (in place, large batches)
#pragma once

#include "common.cuh"

namespace gqa {
namespace tree {

struct CommitParams {
  const int32_t *path, *path_lens, *seq_lens;
  int32_t *lens_out, *status;
  int B, Hkv, C, t_new, P, vpr;  // vpr: vectors per row
};

// Block-wide: every length in [0, C], path lengths in [0, min(P, t_new)]
// that fit behind them, paths strictly ascending inside [0, t_new).  Returns
// 0 or the status of the first kind of fault (capacity before path).
__device__ __forceinline__ int commit_fault(const CommitParams &p) {
  int cap = 0, bad = 0;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int n = p.seq_lens[b], a = p.path_lens[b];
    bad |= a < 0 || a > min(p.P, p.t_new);
    cap |= n < 0 || n > p.C || (a > 0 && a > p.C - n);
  }
  const int64_t total = (int64_t)p.B * p.P;
  for (int64_t i = threadIdx.x; i < total; i += blockDim.x) {
    const int b = (int)(i / p.P), j = (int)(i - (int64_t)b * p.P);
    if (j >= p.path_lens[b]) continue;
    const int x = p.path[i];
    bad |= x < 0 || x >= p.t_new || (j > 0 && p.path[i - 1] >= x);
  }
  if (__syncthreads_or(cap)) return GQA_ERR_CAPACITY;
  if (__syncthreads_or(bad)) return GQA_ERR_TREE;
  return 0;
}

template <typename V>
__global__ void __launch_bounds__(256)
    tree_commit_kernel(V *__restrict__ kc, V *__restrict__ vc, const V *__restrict__ kd,
                       const V *__restrict__ vd, const CommitParams p, int commit, int cluster) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int fault = commit_fault(p);
  if (fault) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_status(p.status, fault);
  } else {
    constexpr int U = 8;
    const int64_t lane_cols = (int64_t)p.B * p.Hkv * p.vpr;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < 2 * lane_cols;
         i += (int64_t)gridDim.x * blockDim.x) {
      const bool isv = i >= lane_cols;
      const int64_t c = isv ? i - lane_cols : i;
      const int64_t lane = c / p.vpr;  // b * Hkv + g
      const int col = (int)(c - lane * p.vpr);
      const int b = (int)(lane / p.Hkv);
      const int n = p.seq_lens[b], a = p.path_lens[b];
      const V *src = (isv ? vd : kd) + lane * p.t_new * p.vpr + col;
      V *dst = (isv ? vc : kc) + (lane * p.C + n) * p.vpr + col;
      const int32_t *path = p.path + (int64_t)b * p.P;
      for (int j0 = 0; j0 < a; j0 += U) {
        V x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j0 + u < a) x[u] = src[(int64_t)path[j0 + u] * p.vpr];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j0 + u < a) dst[(int64_t)(j0 + u) * p.vpr] = x[u];
      }
    }
  }
  if (!commit) return;
  if (cluster) {  // every CTA of the one cluster has read the lengths
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // a refused call leaves the lengths as they are (copied to lens_out)
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += blockDim.x)
      p.lens_out[b] = p.seq_lens[b] + (fault ? 0 : p.path_lens[b]);
}

__global__ void __launch_bounds__(256) tree_commit_lens_kernel(const CommitParams p) {
  griddep_wait();
  if (commit_fault(p)) return;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) p.lens_out[b] = p.seq_lens[b] + p.path_lens[b];
}

}  // namespace tree
}  // namespace gqa
