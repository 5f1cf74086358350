// norm_rope.cu -- gqa_qk_norm_rope: argument checks, choice of kernel, launch.
#include <algorithm>

#include "host.cuh"
#include "norm_rope.cuh"

namespace {

using namespace gqa::host;
using gqa::nr::Params;

// Heads per CTA: all of them (a token's angles are then computed once) while
// that gives every SM a CTA, else halved until it does; a few tokens take a
// head per CTA.  More than 16 heads are halved until every SM has two, since
// their CTAs' unequal numbers then show more than the angles.  bf16, 48 heads
// of 128: 1024 tokens 9.0 us with 12 heads per CTA (256 CTAs), 12.0 with 6,
// 11.6 with 24; 4096 tokens 27.4 with 48, 25.0 with 24, 24.3 with 12; fp32, 12
// heads of 64, 4084 tokens: 6.4 with 12, 7.7 with 6, 8.3 with 3.
int heads_per_cta(int64_t token_ctas, int heads, int sms) {
  int hpg = heads;
  while (hpg > 1) {
    const int64_t ctas = token_ctas * ((heads + hpg - 1) / hpg);
    if (ctas >= (hpg > 16 ? 2 : 1) * (int64_t)sms) break;
    hpg = (hpg + 1) / 2;
  }
  return hpg;
}

template <typename T, int G>
gqa_status launch_vec(Params p, int sms, cudaStream_t st) {
  constexpr int tok = gqa::nr::kThreads / G;
  const int heads = p.Hq + 2 * p.Hkv;
  const int64_t grid = (p.tokens + tok - 1) / tok;
  p.hpg = heads_per_cta(grid, heads, sms);
  const int chunks = (heads + p.hpg - 1) / p.hpg;
  if (grid > INT_MAX || chunks > 65535) return GQA_ERR_UNSUPPORTED;
  const bool part = 2 * p.half < p.d;
  auto *kernel = p.interleaved ? (part ? gqa::nr::norm_rope_vec_kernel<T, G, true, true>
                                       : gqa::nr::norm_rope_vec_kernel<T, G, true, false>)
                               : (part ? gqa::nr::norm_rope_vec_kernel<T, G, false, true>
                                       : gqa::nr::norm_rope_vec_kernel<T, G, false, false>);
  return launched(gqa::launch_dependent(kernel, dim3((unsigned)grid, (unsigned)chunks),
                                        dim3(gqa::nr::kThreads), 0, st, p));
}

template <typename T>
gqa_status launch(const Params &p, bool vec, int sms, cudaStream_t st) {
  constexpr int N = gqa::nr::Vec<T>::N;
  if (vec) {
    if (p.d <= 8 * N) return launch_vec<T, 8>(p, sms, st);
    if (p.d <= 16 * N) return launch_vec<T, 16>(p, sms, st);
    return launch_vec<T, 32>(p, sms, st);
  }
  const int64_t rows = p.tokens * (p.Hq + 2 * p.Hkv);
  const int64_t grid = std::min<int64_t>((rows + 7) / 8, (int64_t)sms * 8);
  return launched(gqa::launch_dependent(gqa::nr::norm_rope_row_kernel<T>, dim3((unsigned)grid),
                                        dim3(gqa::nr::kThreads), 0, st, p));
}

}  // namespace

extern "C" gqa_status gqa_qk_norm_rope(
    gqa_dtype dtype, const void *qkv, int64_t batch_stride, int64_t row_stride,
    const void *q_weight, const void *k_weight, float eps, const float *inv_freq, int rot_d,
    int interleaved, const int32_t *positions, int axes, const int32_t *pair_axis, void *q,
    void *k, void *v, int B, int Hq, int Hkv, int T, int d, gqa_stream_t stream) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_UNSUPPORTED;
  if (B < 0 || T < 0) return GQA_ERR_SHAPE;
  gqa_status s = check_heads(Hq, Hkv, d);
  if (s != GQA_OK) return s;
  if (rot_d < 0 || rot_d > d || (rot_d & 1)) return GQA_ERR_SHAPE;
  if (!(eps >= 0.f)) return GQA_ERR_SHAPE;
  int64_t heads = (int64_t)Hq + 2 * (int64_t)Hkv, width, n, pos;
  if (!elems(&width, {heads, d}) || !elems(&n, {B, T, width}) || n > INT64_MAX / 8 ||
      !elems(&pos, {std::max(axes, 0), B, T}))
    return GQA_ERR_OVERFLOW;
  if (heads > INT_MAX / 2) return GQA_ERR_OVERFLOW;
  if (row_stride < width || batch_stride < 0) return GQA_ERR_SHAPE;
  int64_t span;
  if (!elems(&span, {std::max(T - 1, 0), row_stride}) || span > INT64_MAX / 16 ||
      !elems(&span, {std::max(B - 1, 0), batch_stride}) || span > INT64_MAX / 16)
    return GQA_ERR_OVERFLOW;
  if (axes < 1 || axes > gqa::nr::kMaxAxes) return GQA_ERR_SHAPE;
  Params p = {};
  if (pair_axis)
    for (int i = 0; i < rot_d / 2 && i < 128; ++i) {
      if (pair_axis[i] < 0 || pair_axis[i] >= axes) return GQA_ERR_SHAPE;
      p.axis[i >> 4] |= (uint32_t)pair_axis[i] << (2 * (i & 15));
    }
  if (B == 0 || T == 0) return GQA_OK;
  if (!qkv || !q || !k || !v) return GQA_ERR_NULL;
  if (rot_d > 0 && !inv_freq) return GQA_ERR_NULL;
  if (axes > 1 && !positions) return GQA_ERR_NULL;
  if (d > GQA_MAX_HEAD_DIM) return GQA_ERR_UNSUPPORTED;
  DeviceInfo di;
  if ((s = device_info(&di)) != GQA_OK) return s;
  p.qkv = qkv;
  p.qw = q_weight;
  p.kw = k_weight;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.q = q;
  p.k = k;
  p.v = v;
  p.batch_stride = batch_stride;
  p.row_stride = row_stride;
  p.tokens = (int64_t)B * T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.T = T;
  p.d = d;
  p.half = rot_d / 2;
  p.interleaved = interleaved ? 1 : 0;
  p.eps = eps;
  p.inv_d = 1.f / (float)d;
  // 16-byte vectors: rows of whole vectors, at most 32 of them, all aligned,
  // and pairs (i, i + half) at the same place of two lanes' vectors
  const int N = dtype == GQA_F32 ? 4 : 8;
  const bool vec = d % N == 0 && d <= 32 * N && row_stride % N == 0 && batch_stride % N == 0 &&
                   (interleaved || p.half % N == 0) && aligned16(qkv) && aligned16(q) &&
                   aligned16(k) && aligned16(v);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == GQA_F32 ? launch<float>(p, vec, di.sms, st)
                          : launch<__nv_bfloat16>(p, vec, di.sms, st);
}
