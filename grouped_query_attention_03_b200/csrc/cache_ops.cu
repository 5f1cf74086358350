// cache_ops.cu -- gqa_tree_commit and gqa_cache_evict: argument checks and
// launches.
#include <algorithm>

#include "evict.cuh"
#include "host.cuh"
#include "tree_commit.cuh"

namespace {

using namespace gqa::host;
using gqa::evict::kMaxCluster;

// Vectors a row is moved in: 16 bytes where rows and buffers allow, else
// elements.
struct RowVec {
  int bytes;  // of one vector
  int vpr;    // vectors per row
};

RowVec row_vec(gqa_dtype dtype, int d, std::initializer_list<const void *> ptrs) {
  const int esz = dtype == GQA_F32 ? 4 : 2;
  bool ok = (int64_t)d * esz % 16 == 0;
  for (const void *p : ptrs) ok = ok && aligned16(p);
  return ok ? RowVec{16, d * esz / 16} : RowVec{esz, d};
}

// Columns a tree commit moves with one cluster of 8 CTAs; larger in-place
// commits take the whole GPU and a second launch for the lengths (2048
// columns, 8 lanes of 8 sequences: 5.3 us against 6.6; 4096: 6.6 both; 8192:
// 9.1 against 7.5).
constexpr int64_t kClusterCols = 4096;

template <typename V>
gqa_status launch_commit(void *kc, void *vc, const void *kd, const void *vd,
                         gqa::tree::CommitParams p, int sms, cudaStream_t st) {
  const int64_t cols = (int64_t)2 * p.B * p.Hkv * p.vpr;
  const bool apart = p.lens_out != p.seq_lens;
  const bool cluster = !apart && cols <= kClusterCols;
  const int64_t want = (cols + 255) / 256;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cluster ? std::min<int64_t>(want, 8)
                                        : std::min<int64_t>(want, (int64_t)sms * 8)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cfg.gridDim.x;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  const int commit = apart || cluster ? 1 : 0;
  gqa_status s = launched(cudaLaunchKernelEx(&cfg, gqa::tree::tree_commit_kernel<V>, (V *)kc,
                                             (V *)vc, (const V *)kd, (const V *)vd, p, commit,
                                             cluster ? 1 : 0));
  if (s != GQA_OK || commit) return s;
  return launched(gqa::launch_dependent(gqa::tree::tree_commit_lens_kernel, dim3(1), dim3(256), 0,
                                        st, p));
}

template <int KPT>
gqa_status launch_select_k(const gqa::evict::Params &p, int cluster, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)p.B * p.Hkv * cluster));
  cfg.blockDim = dim3(gqa::evict::kSelThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return launched(cudaLaunchKernelEx(&cfg, gqa::evict::evict_select_kernel<KPT>, p, cluster));
}

// CTAs per lane.  A cluster's launch, barriers and remote counts cost more
// than reading a few thousand cells does (8 lanes of 4000 cells, to 2048:
// 10.2 us with a CTA each, 11.4 with two, 13.8 with four, 18.2 with eight), so
// a CTA gets at least 8 strips of 512 cells, and a cluster up to 4 of them
// while the lanes leave SMs for more (8 lanes of 32768 cells, to 4096: 42 us
// with one, 20.8 with two, 17.9 with four, 25.5 with eight; 64 lanes of 8000,
// to 4096: 57.4, 56.4, 58.1).  Longer lanes take as many CTAs, up to 8, as
// hold their keys in registers (32 a thread); a lane that 8 cannot hold is
// read again for every digit by one.
gqa_status launch_select(const gqa::evict::Params &p, int sms, cudaStream_t st) {
  using namespace gqa::evict;
  const int64_t lanes = (int64_t)p.B * p.Hkv;
  const int64_t strips = ((int64_t)p.C + kSelThreads - 1) / kSelThreads;
  int cluster = 1;
  while (cluster < kMaxCluster &&
         ((cluster < 4 && strips > 8 * cluster && lanes * cluster * 2 <= sms) ||
          strips > 32 * cluster))
    cluster *= 2;
  const int64_t kpt = (strips + cluster - 1) / cluster;
  if (lanes * cluster > INT_MAX) return GQA_ERR_UNSUPPORTED;
  if (kpt <= 4) return launch_select_k<4>(p, cluster, st);
  if (kpt <= 8) return launch_select_k<8>(p, cluster, st);
  if (kpt <= 16) return launch_select_k<16>(p, cluster, st);
  if (kpt <= 32) return launch_select_k<32>(p, cluster, st);
  return launch_select_k<0>(p, 1, st);
}

template <typename V>
gqa_status launch_evict_rows(const void *kc, const void *vc, void *ko, void *vo,
                             const gqa::evict::Params &p, int vpr, bool in_place, int sms,
                             cudaStream_t st) {
  if (in_place) {
    // slices of 64 bytes (4 vectors): a whole DRAM burst each, and 8 CTAs a
    // lane for a 256-byte row of K and V
    constexpr int SL = sizeof(V) == 16 ? 4 : 32;
    const int slices = (vpr + SL - 1) / SL;
    const int64_t grid = (int64_t)p.B * p.Hkv * 2 * slices;
    if (grid > INT_MAX) return GQA_ERR_UNSUPPORTED;
    return launched(gqa::launch_dependent(gqa::evict::evict_move_kernel<V, SL>,
                                          dim3((unsigned)grid), dim3(256), 0, st, (V *)ko,
                                          (V *)vo, p, vpr, slices));
  }
  const int64_t total = (int64_t)p.B * p.Hkv * p.budget * vpr;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((total + 1023) / 1024, (int64_t)sms * 8));
  return launched(gqa::launch_dependent(gqa::evict::evict_copy_kernel<V>, dim3((unsigned)grid),
                                        dim3(256), 0, st, (const V *)kc, (const V *)vc, (V *)ko,
                                        (V *)vo, p, vpr));
}

}  // namespace

extern "C" {

gqa_status gqa_tree_commit(gqa_dtype dtype, void *k_cache, void *v_cache, const void *k_draft,
                           const void *v_draft, const int32_t *path, const int32_t *path_lens,
                           const int32_t *seq_lens, int32_t *lens_out, int B, int Hkv, int C,
                           int d, int t_new, int max_path, int32_t *dev_status,
                           gqa_stream_t stream) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_UNSUPPORTED;
  if (B < 0 || C < 0 || t_new < 0 || max_path < 0) return GQA_ERR_SHAPE;
  if (Hkv <= 0 || d <= 0) return GQA_ERR_SHAPE;
  int64_t nc, nd, np, cols;
  if (!elems(&nc, {B, Hkv, C, d}) || !elems(&nd, {B, Hkv, t_new, d}) ||
      !elems(&np, {B, max_path}) || !elems(&cols, {B, Hkv, d, 8}) || nc > INT64_MAX / 8 ||
      nd > INT64_MAX / 8 || d > INT_MAX / 8)
    return GQA_ERR_OVERFLOW;
  if (B == 0) return GQA_OK;
  if (!path_lens || !seq_lens || !lens_out || !dev_status) return GQA_ERR_NULL;
  if (C > 0 && (!k_cache || !v_cache)) return GQA_ERR_NULL;
  if (t_new > 0 && max_path > 0 && (!k_draft || !v_draft || !path)) return GQA_ERR_NULL;
  DeviceInfo di;
  gqa_status s = device_info(&di);
  if (s != GQA_OK) return s;
  const RowVec rv = row_vec(dtype, d, {k_cache, v_cache, k_draft, v_draft});
  gqa::tree::CommitParams p;
  p.path = path;
  p.path_lens = path_lens;
  p.seq_lens = seq_lens;
  p.lens_out = lens_out;
  p.status = dev_status;
  p.B = B;
  p.Hkv = Hkv;
  p.C = C;
  p.t_new = t_new;
  p.P = max_path;
  p.vpr = rv.vpr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rv.bytes == 16)
    return launch_commit<uint4>(k_cache, v_cache, k_draft, v_draft, p, di.sms, st);
  if (rv.bytes == 4)
    return launch_commit<uint32_t>(k_cache, v_cache, k_draft, v_draft, p, di.sms, st);
  return launch_commit<uint16_t>(k_cache, v_cache, k_draft, v_draft, p, di.sms, st);
}

gqa_status gqa_cache_evict(gqa_dtype dtype, const void *k_cache, const void *v_cache,
                           const float *weights, const int32_t *seq_lens, void *k_out,
                           void *v_out, float *weights_out, int32_t *lens_out, int32_t *kept,
                           int B, int Hkv, int C, int C_out, int d, int budget, int recent,
                           int32_t *dev_status, gqa_stream_t stream) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_UNSUPPORTED;
  if (B < 0 || C < 0 || C_out < 0 || budget < 0 || recent < 0) return GQA_ERR_SHAPE;
  if (Hkv <= 0 || d <= 0) return GQA_ERR_SHAPE;
  if (recent > budget || budget > C_out) return GQA_ERR_CAPACITY;
  int64_t nc, no;
  if (!elems(&nc, {B, Hkv, C, d}) || !elems(&no, {B, Hkv, C_out, d}) || nc > INT64_MAX / 8 ||
      no > INT64_MAX / 8 || d > INT_MAX / 8)
    return GQA_ERR_OVERFLOW;
  if (B == 0) return GQA_OK;
  // nothing to read, or nothing to keep and no weights to clear: the lengths
  // are still to be written, so the kernels run
  if (!seq_lens || !lens_out || !dev_status) return GQA_ERR_NULL;
  if (C > 0 && (!k_cache || !v_cache || !weights)) return GQA_ERR_NULL;
  if (C_out > 0 && (!k_out || !v_out || !weights_out)) return GQA_ERR_NULL;
  if (budget > 0 && !kept) return GQA_ERR_NULL;
  // in place: all three buffers, and of the same capacity
  const bool in_place = k_out == k_cache;
  if ((v_out == v_cache) != in_place || (weights_out == weights) != in_place ||
      (in_place && C != C_out))
    return GQA_ERR_SHAPE;
  if (C > (1 << 30) || C_out > (1 << 30)) return GQA_ERR_UNSUPPORTED;
  // grids (a lane's cluster, its column slices), before anything is enqueued
  int64_t blocks;
  if (!elems(&blocks, {B, Hkv, std::max(kMaxCluster, 2 * (d / 4 + 1))}) || blocks > INT_MAX)
    return GQA_ERR_UNSUPPORTED;
  DeviceInfo di;
  gqa_status s = device_info(&di);
  if (s != GQA_OK) return s;
  gqa::evict::Params p;
  p.w = weights;
  p.w_out = weights_out;
  p.seq_lens = seq_lens;
  p.lens_out = lens_out;
  p.kept = kept;
  p.status = dev_status;
  p.B = B;
  p.Hkv = Hkv;
  p.C = C;
  p.C_out = C_out;
  p.budget = budget;
  p.recent = recent;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if ((s = launch_select(p, di.sms, st)) != GQA_OK) return s;
  const RowVec rv = row_vec(dtype, d, {k_cache, v_cache, k_out, v_out});
  if (rv.bytes == 16)
    return launch_evict_rows<uint4>(k_cache, v_cache, k_out, v_out, p, rv.vpr, in_place, di.sms, st);
  if (rv.bytes == 4)
    return launch_evict_rows<uint32_t>(k_cache, v_cache, k_out, v_out, p, rv.vpr, in_place, di.sms, st);
  return launch_evict_rows<uint16_t>(k_cache, v_cache, k_out, v_out, p, rv.vpr, in_place, di.sms, st);
}

}  // extern "C"
