// decode_host.cuh -- host side of the split-K decode kernel, shared by
// gqa_decode and its relatives and by gqa_decode_scored: plan, workspace
// layout, launch.
#pragma once

#include <algorithm>

#include "decode_splitk.cuh"
#include "host.cuh"
#include "tma_host.cuh"

namespace gqa {
namespace dechost {

using namespace host;
using dec::kLensSmem;
using dec::split_kernel;

constexpr int kMaxDecodeCtas = dec::kMaxCtas;  // workspace is sized for this many
#ifndef GQA_DEC_MIN_ROWS
#define GQA_DEC_MIN_ROWS 320
#endif
// Smallest row range per CTA: small calls use fewer CTAs, so that a lane is
// split into at most about 16 partials, which the merge reads in one batch
// (swept 256-384 on the 16.8 MB sliding-window step: 320 fastest).
constexpr int kDecodeMinRows = GQA_DEC_MIN_ROWS;
#ifndef GQA_DEC_LANE_PAD_BYTES
#define GQA_DEC_LANE_PAD_BYTES 131072
#endif
// A lane segment's fixed cost in a CTA, as cache bytes: the split gives each
// non-empty lane this many bytes of virtual rows (see dec::extent).
constexpr int kDecodeLanePadBytes = GQA_DEC_LANE_PAD_BYTES;

inline int next_pow2(int x) {
  int p = 1;
  while (p < x) p <<= 1;
  return p;
}

// ------------------------------------------------------------ decode plan
struct DecPlan {
  int R = 1;     // heads stacked per CTA lane (power of two, <= 16)
  int nsub = 1;  // sub-groups per KV head
  int VL = 1;    // virtual lanes per batch row
};

inline DecPlan decode_plan(int Hq, int Hkv) {
  DecPlan p;
  const int r = Hq / Hkv;
  p.R = r >= 16 ? 16 : next_pow2(r);
  p.nsub = (r + p.R - 1) / p.R;
  p.VL = Hkv * p.nsub;
  return p;
}

struct DecLayout {
  size_t counters = 0, ml = 0, acc = 0, total = 0;
  size_t counter_bytes = 0;
};

// Workspace: the arrival counters (one per possible first CTA of a split
// lane, and one count of CTAs that have read the lengths) at a fixed place
// for every shape, zero between calls; then the (m, l) and acc partials, one
// slot per (lane, CTA) pair touching it.
inline bool decode_layout(int B, int Hq, int Hkv, int d, DecLayout *L) {
  const DecPlan pl = decode_plan(Hq, Hkv);
  int64_t lanes, slots, ml_elems, acc_elems;
  if (!elems(&lanes, {B, pl.VL})) return false;
  slots = lanes + kMaxDecodeCtas;
  if (!elems(&ml_elems, {slots, pl.R})) return false;
  if (!elems(&acc_elems, {slots, pl.R, d})) return false;
  if (acc_elems > INT64_MAX / 8) return false;
  L->counters = 0;
  L->counter_bytes = (size_t)(gqa::dec::kCtrFinish + 1) * sizeof(int);
  L->ml = round256(L->counter_bytes);
  L->acc = L->ml + round256((size_t)ml_elems * sizeof(float2));
  L->total = L->acc + round256((size_t)acc_elems * sizeof(float));
  return true;
}

inline bool splitk_supported(gqa_dtype dtype, int d) {
  return dtype == GQA_BF16 && (d == 64 || d == 128);
}

// The split-K kernel addresses cache rows with 32-bit TMA coordinates.
inline bool splitk_rows_ok(int B, int Hkv, int C) {
  return (long long)B * Hkv * C < (1LL << 31);
}

// (static: a program may hold two builds of the library, each with its own
// kernels and launch state)
template <int D, int R, bool SC>
static gqa_status launch_splitk(const gqa::dec::Params &p, const void *k_cache,
                         const void *v_cache, int sms, cudaStream_t st) {
  using K = gqa::dec::Cfg<D, R>;
  CUtensorMap mk, mv;
  const long long rows = (long long)p.B * p.Hkv * p.C;
  if (!gqa::tma::make_bf16_map(&mk, k_cache, D, rows, 0, K::ROWS) ||
      !gqa::tma::make_bf16_map(&mv, v_cache, D, rows, 0, K::ROWS))
    return GQA_ERR_CUDA;
  static bool done[64] = {};
  DeviceInfo di;
  gqa_status s = device_info(&di);
  if (s == GQA_OK)
    s = allow_smem(split_kernel<D, R, SC>, K::SMEM + kLensSmem * 4, di.id, done);
  if (s != GQA_OK) return s;
  const int grid = std::min(kMaxDecodeCtas, K::MIN_BLOCKS * sms);
  // the lengths' shared-memory copy follows the stages
  const int smem = K::SMEM + (p.lens_smem ? ((p.B * 4 + 15) & ~15) : 0);
  // A programmatic dependent of the previous kernel on the stream: its CTAs
  // set up while that kernel drains and wait for it before touching memory.
  if (gqa::launch_dependent(split_kernel<D, R, SC>, dim3(grid), dim3(K::THREADS), smem,
                            st, mk, mv, p) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return launch_status();
}

template <int D, bool SC = false>
static gqa_status dispatch_splitk_R(int R, const gqa::dec::Params &p, const void *kc,
                             const void *vc, int sms, cudaStream_t st) {
  switch (R) {
    case 1: return launch_splitk<D, 1, SC>(p, kc, vc, sms, st);
    case 2: return launch_splitk<D, 2, SC>(p, kc, vc, sms, st);
    case 4: return launch_splitk<D, 4, SC>(p, kc, vc, sms, st);
    case 8: return launch_splitk<D, 8, SC>(p, kc, vc, sms, st);
    case 16: return launch_splitk<D, 16, SC>(p, kc, vc, sms, st);
  }
  return GQA_ERR_UNSUPPORTED;
}

}  // namespace dechost
}  // namespace gqa
