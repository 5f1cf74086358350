// rows.cu -- gqa_decode_tree and gqa_decode_scored: argument checks, the
// workspace, the choice of kernel, launches.
#include <algorithm>

#include "decode_host.cuh"
#include "host.cuh"
#include "rows_simt.cuh"
#include "rows_splitk.cuh"
#include "rows_weigh_tc.cuh"

namespace {

using namespace gqa::host;
using gqa::rows::Params;

// The workspace is sized for this many CTAs of the tensor-core kernel (one
// per SM), and the CUDA-core kernel's parts aim at this many CTAs, so that
// neither depends on the device.
constexpr int kMaxCtas = 256;
constexpr int kSimtCtas = 592;
// Keys that a part of the CUDA-core kernel has at least (fp32, one head of 64, 44
// nodes, 482 cells: 18.3 us with 64, 21.6 with 128; 16 groups of 4 rows over
// 1000 cells: 26.5 and 22.6; in between elsewhere).
constexpr int kPartKeys = 64;

// What a lane group costs a CTA besides its tiles, in tiles (64 ragged
// sequences, 63 nodes: 120 us with 2, 111 with 3 and with 4, 114 with 5).
constexpr int kPadTiles = 3;

// Rows times parts that the last CTA to count a lane group's parts merges
// itself; more than that is shared by all SMs in a kernel of its own (d = 128,
// r = 4: 8 sequences of 8000 cells, 26 nodes, 4 parts: 56 us, 63 with the
// kernel; 2 sequences, 8 nodes, 10 parts: 25.1 us with it, 27.9 without; one of
// 1000 cells: 13.3 and 19.5).
constexpr int kMergeRows = 800;

// Parts that a warp of that kernel merges alone; more are shared by four (2 lanes
// of 53 rows, 62 parts: 13.9 us with the attention, 24.3 alone; 2 of 256 rows, 74
// parts: 30.1 and 35.5; but 8 lanes of 64 rows, 18 parts: 17.3 and 16.3).
constexpr int kPartsPerWarp = 32;

// Calls that share a workspace find each other's counters at the same place.
static_assert(gqa::rows::kCounters == gqa::dec::kCtrFinish, "the counters' region");
static_assert((gqa::rows::kCounters + 1) * sizeof(int) <= GQA_WORKSPACE_ZERO_BYTES, "what must be zero");

struct Layout {
  bool tc = false;
  bool dec = false;     // scored, one row: the decode kernel
  bool finish = false;  // the parts are merged by a kernel of their own
  bool scores = false;  // scored: the scores are kept, not multiplied again
  int part_warps = 1;   // that share a lane group's parts in the merge
  int NT = 1, group_rows = 0, MG = 1, ns = 0, Cp = 0;
  int64_t slots = 0;
  size_t groups = 0, ml = 0, acc = 0, lse = 0, score_at = 0, total = 0;  // counters at 0
};

// Sizes only (no pointers): what gqa_decode_*_workspace_bytes can know.  The
// tensor-core kernel addresses query rows with 32-bit TMA coordinates.
bool layout(gqa_dtype dtype, int B, int Hq, int Hkv, int C, int d, int t, bool scored, bool tc_ok,
            Layout *out) {
  Layout L;
  int64_t R, rows, lanes, x;
  if (!elems(&R, {Hq / Hkv, t}) || !elems(&rows, {B, Hq, t}) || !elems(&lanes, {B, Hkv}))
    return false;
  if (rows > INT_MAX / 2 || lanes > INT_MAX / 2) return false;
  const bool tc_type = dtype == GQA_BF16 && (d == 64 || d == 128);
  L.tc = tc_ok && tc_type;
  // With many rows the tensor-core kernel's scores are not kept but multiplied
  // again (8 lanes of 32768 cells, d = 128: 32 rows 53.8 us with the scores kept,
  // 59.0 with the keys read again; 64 rows 74.6 and 60.5).  Nor are they where
  // the buffers' alignment sends such a call to CUDA cores, so that a workspace
  // holds them only where they are always used.
  L.scores = scored && !(tc_type && R > d / 4);
  // One scored row is a decode step: its kernel reads the cache at the same
  // rate and has a tenth of the tile kernel's fixed costs (B = 8, 8001 cells:
  // 59 us with tiles of 128 rows).  Within that kernel's limits, those of
  // gqa_decode; the tiles have none of them.
  L.dec = L.tc && scored && t == 1 && gqa::dechost::splitk_rows_ok(B, Hkv, C) && B <= 65535 &&
          gqa::dechost::decode_plan(Hq, Hkv).VL <= 65535;
  if (L.dec) {
    gqa::dechost::DecLayout D;
    if (!gqa::dechost::decode_layout(B, Hq, Hkv, d, &D)) return false;
    L.ml = D.ml;  // (counters at 0)
    L.acc = D.acc;
    L.lse = round256(D.total);
    L.scores = true;  // (of one row each, whatever the group)
  } else if (L.tc) {
    // up to 128 rows fill one row tile; more are taken in pairs of tiles, so
    // that two share each K and V tile
    L.NT = R <= gqa::rows::kM ? 1 : 2;
    L.MG = (int)((R + 2 * gqa::rows::kM - 1) / (2 * gqa::rows::kM));
    L.group_rows = L.MG == 1 ? (int)R : 2 * gqa::rows::kM;
    L.slots = lanes * L.MG + kMaxCtas;
    // Parts per lane group if all sequences are of one length, and their rows:
    // what the last CTA to count them would have to read.
    const int64_t parts = kMaxCtas / 2 / std::max<int64_t>(lanes * L.MG, 1) + 2;
    L.part_warps = parts > kPartsPerWarp ? 4 : 1;
    L.finish = parts > gqa::rows::kAddParts || parts * L.group_rows > kMergeRows;
  } else {
    L.group_rows = gqa::rows::kSR;
    L.MG = (int)((R + gqa::rows::kSR - 1) / gqa::rows::kSR);
    // parts of at least kPartKeys keys, enough of them to fill the GPU
    const int64_t groups = lanes * L.MG;
    const int64_t most = std::max<int64_t>(1, ((int64_t)C + t) / kPartKeys);
    L.ns = (int)std::min<int64_t>(std::min<int64_t>(most, 64),
                                  std::max<int64_t>(1, kSimtCtas / std::max<int64_t>(groups, 1)));
    L.slots = groups * L.ns;
  }
  if (!L.dec) {
    int64_t n;
    // (one more counter than are used here: the decode kernel's region)
    L.groups = round256((gqa::rows::kCounters + 1) * sizeof(int));
    L.ml = L.groups + (L.finish ? round256((size_t)(lanes * L.MG) * sizeof(int2)) : 0);
    if (!elems(&n, {L.slots, L.group_rows, 8}) || n > INT64_MAX / 8) return false;
    L.acc = L.ml + round256((size_t)n);
    if (!elems(&n, {L.slots, L.group_rows, (d + 3) / 4, 16}) || n > INT64_MAX / 8) return false;
    L.lse = L.acc + round256((size_t)n);
  }
  L.total = L.lse;
  if (scored) {
    if (!elems(&x, {lanes, R, 8}) || x > INT64_MAX / 8) return false;
    L.score_at = L.lse + round256((size_t)x);
    L.total = L.score_at;
    if (C > INT_MAX - gqa::rows::kTile) return false;
    L.Cp = (C + gqa::rows::kTile - 1) / gqa::rows::kTile * gqa::rows::kTile;
    if (L.scores) {
      if (!elems(&x, {lanes, R, L.Cp, 4}) || x > INT64_MAX / 8) return false;
      L.total += round256((size_t)x);
    }
  }
  *out = L;
  return true;
}

template <int D, int NT>
gqa_status launch_tc(const Params &p, const DeviceInfo &di, cudaStream_t st) {
  using K = gqa::rows::TcCfg<D, NT>;
  CUtensorMap mq, mk, mv, mkd, mvd;
  const int lanes = p.B * p.Hkv;
  // a lane's rows are consecutive; those past them read as zeros
  if (!gqa::tma::make_bf16_map(&mq, p.q, D, p.R, lanes, 128)) return GQA_ERR_CUDA;
  if (p.C > 0 && (!gqa::tma::make_bf16_map(&mk, p.k, D, p.C, lanes, 128) ||
                  !gqa::tma::make_bf16_map(&mv, p.v, D, p.C, lanes, 128)))
    return GQA_ERR_CUDA;
  if (p.tree && (!gqa::tma::make_bf16_map(&mkd, p.kd, D, p.t, lanes, 128) ||
                 !gqa::tma::make_bf16_map(&mvd, p.vd, D, p.t, lanes, 128)))
    return GQA_ERR_CUDA;
  // a map that no tile uses stands for its pair
  if (p.C == 0) {
    mk = mkd;
    mv = mvd;
  }
  if (!p.tree) {
    mkd = mk;
    mvd = mv;
  }
  static bool done[64] = {};
  gqa_status s = allow_smem(gqa::rows::rows_splitk_kernel<D, NT>, K::SMEM, di.id, done);
  if (s != GQA_OK) return s;
  return launched(gqa::launch_dependent(gqa::rows::rows_splitk_kernel<D, NT>,
                                        dim3((unsigned)p.ctas), dim3(gqa::rows::kTcThreads), K::SMEM, st, mq,
                                        mk, mv, mkd, mvd, p));
}

template <int D>
gqa_status launch_weigh_tc(const Params &p, const DeviceInfo &di, cudaStream_t st) {
  using K = gqa::rows::WgCfg<D>;
  CUtensorMap mq, mk;
  if (!gqa::tma::make_bf16_map(&mq, p.q, D, p.R, p.B * p.Hkv, 128) ||
      !gqa::tma::make_bf16_map(&mk, p.k, D, p.C, p.B * p.Hkv, 128))
    return GQA_ERR_CUDA;
  static bool done[64] = {};
  gqa_status s = allow_smem(gqa::rows::rows_weigh_tc_kernel<D>, K::SMEM, di.id, done);
  if (s != GQA_OK) return s;
  return launched(gqa::launch_dependent(gqa::rows::rows_weigh_tc_kernel<D>,
                                        dim3((unsigned)di.sms), dim3(gqa::rows::kTcThreads),
                                        K::SMEM, st, mq, mk, p));
}

template <typename T, int RPT>
gqa_status launch_simt_rpt(const Params &p, const DeviceInfo &di, cudaStream_t st) {
  const int64_t grid = (int64_t)p.B * p.Hkv * p.MG * p.ns;
  if (grid > INT_MAX) return GQA_ERR_UNSUPPORTED;
  static bool done[64] = {};
  gqa_status s = allow_smem(gqa::rows::rows_simt_kernel<T, RPT>,
                            gqa::rows::simt_smem(GQA_MAX_HEAD_DIM, sizeof(T)), di.id, done);
  if (s != GQA_OK) return s;
  return launched(gqa::launch_dependent(gqa::rows::rows_simt_kernel<T, RPT>, dim3((unsigned)grid),
                                        dim3(gqa::rows::kSimtThreads),
                                        gqa::rows::simt_smem(p.d, sizeof(T)), st, p));
}

template <typename T>
gqa_status launch_simt(Params p, const DeviceInfo &di, cudaStream_t st) {
  p.vec = p.d * (int)sizeof(T) % 16 == 0 && aligned16(p.k) && aligned16(p.v) && aligned16(p.kd) &&
          aligned16(p.vd);
  switch (gqa::rows::simt_rpt(p.d)) {
    case 1: return launch_simt_rpt<T, 1>(p, di, st);
    case 2: return launch_simt_rpt<T, 2>(p, di, st);
    case 4: return launch_simt_rpt<T, 4>(p, di, st);
    default: return launch_simt_rpt<T, 8>(p, di, st);
  }
}

// One row per sequence on the decode kernel, scores and statistics kept.
gqa_status launch_dec(const Params &p, const Layout &L, const DeviceInfo &di, cudaStream_t st) {
  const gqa::dechost::DecPlan pl = gqa::dechost::decode_plan(p.Hq, p.Hkv);
  gqa::dec::Params x = {};
  x.q = (const __nv_bfloat16 *)p.q;
  x.o = (__nv_bfloat16 *)p.o;
  x.seq_lens = p.seq_lens;
  x.B = p.B;
  x.Hq = p.Hq;
  x.Hkv = p.Hkv;
  x.C = p.C;
  x.window = GQA_NO_WINDOW;
  x.scale_log2 = p.scale_log2;
  x.r = p.r;
  x.nsub = pl.nsub;
  x.VL = pl.VL;
  x.min_rows = gqa::dechost::kDecodeMinRows;
  x.counters = p.counters;
  x.ml = p.ml;
  x.acc = p.acc;
  x.status = p.status;
  x.lens_smem = p.B <= gqa::dec::kLensSmem ? 1 : 0;
  x.pad = gqa::dechost::kDecodeLanePadBytes / (4 * p.d);  // K and V rows of d bf16
  x.scores = p.scores;
  x.lse = p.lse;
  x.Cp = p.Cp;
  return p.d == 64
             ? gqa::dechost::dispatch_splitk_R<64, true>(pl.R, x, p.k, p.v, di.sms, st)
             : gqa::dechost::dispatch_splitk_R<128, true>(pl.R, x, p.k, p.v, di.sms, st);
}

struct Operands {
  const void *q, *k, *v, *kd, *vd;
  const int32_t *parents, *seq_lens;
  void *o;
  float *weights;  // scored
};

gqa_status rows_impl(gqa_dtype dtype, const Operands &op, bool tree, int B, int Hq, int Hkv, int C,
                     int d, int t, int window, float scale, void *workspace,
                     size_t workspace_bytes, int32_t *dev_status, gqa_stream_t stream) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return GQA_ERR_UNSUPPORTED;
  if (B < 0 || C < 0 || t < 0) return GQA_ERR_SHAPE;
  gqa_status s = check_heads(Hq, Hkv, d);
  if (s != GQA_OK) return s;
  if ((s = check_window(window)) != GQA_OK) return s;
  int64_t nq, nc;
  if (!elems(&nq, {B, Hq, t, d}) || !elems(&nc, {B, Hkv, C, d}) || nq > INT64_MAX / 8 ||
      nc > INT64_MAX / 8)
    return GQA_ERR_OVERFLOW;
  if (t > GQA_MAX_TREE) return GQA_ERR_UNSUPPORTED;
  if (!tree && t > C) return GQA_ERR_CAPACITY;
  if (B == 0 || t == 0) return GQA_OK;
  if (!op.q || !op.o || !op.seq_lens || !dev_status) return GQA_ERR_NULL;
  if (C > 0 && (!op.k || !op.v)) return GQA_ERR_NULL;
  if (tree ? (!op.kd || !op.vd) : !op.weights) return GQA_ERR_NULL;
  if (d > GQA_MAX_HEAD_DIM) return GQA_ERR_UNSUPPORTED;
  const bool aligned = aligned16(op.q) && aligned16(op.k) && aligned16(op.v) && aligned16(op.kd) &&
                       aligned16(op.vd) && aligned16(op.o);
  // tile coordinates and key indexes are 32-bit
  if (C > INT_MAX - 2 * GQA_MAX_TREE) return GQA_ERR_UNSUPPORTED;
  Layout L;
  if (!layout(dtype, B, Hq, Hkv, C, d, t, !tree, aligned, &L)) return GQA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < L.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return GQA_ERR_WORKSPACE;
  DeviceInfo di;
  if ((s = device_info(&di)) != GQA_OK) return s;
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  Params p = {};
  p.q = op.q;
  p.k = op.k;
  p.v = op.v;
  p.kd = op.kd;
  p.vd = op.vd;
  p.parents = op.parents;
  p.seq_lens = op.seq_lens;
  p.o = op.o;
  p.status = dev_status;
  p.counters = reinterpret_cast<int *>(ws);
  p.groups = reinterpret_cast<int2 *>(ws + L.groups);
  p.finish = L.finish ? 1 : 0;
  p.ml = reinterpret_cast<float2 *>(ws + L.ml);
  p.acc = reinterpret_cast<float *>(ws + L.acc);
  p.lse = tree ? nullptr : reinterpret_cast<float2 *>(ws + L.lse);
  p.scores = L.scores ? reinterpret_cast<float *>(ws + L.score_at) : nullptr;
  p.weights = op.weights;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.C = C;
  p.d = d;
  p.t = t;
  p.r = Hq / Hkv;
  p.R = p.r * t;
  p.window = window;
  p.tree = tree ? 1 : 0;
  p.Cp = L.Cp;
  p.group_rows = L.group_rows;
  p.MG = L.MG;
  p.ctas = std::min(kMaxCtas, di.sms);
  p.pad = kPadTiles;
  p.ns = L.ns;
  if (window > 0 && L.ns > 0)  // fewer parts where the window leaves few keys
    p.ns = std::max(1, std::min(L.ns, (std::min(C, window - 1) + t) / kPartKeys));
  p.scale_log2 = scale * gqa::kLog2e;
  // the grids of the kernels that follow, checked before anything is launched
  const int row_blocks =
      (std::min(L.group_rows, p.R) + gqa::rows::kFinishRows - 1) / gqa::rows::kFinishRows;
  const int col_blocks = std::max(1, d / (4 * gqa::rows::kFinishWarps / L.part_warps));
  const int64_t finish_blocks = (int64_t)B * Hkv * L.MG * row_blocks * col_blocks;
  if (L.finish && finish_blocks > INT_MAX) return GQA_ERR_UNSUPPORTED;
  const int per_block = L.scores ? gqa::rows::kWeighCells : gqa::rows::kWeighKeys;
  const int cell_blocks = (C + per_block - 1) / per_block;
  const int64_t grid = tree ? 0 : (int64_t)B * Hkv * cell_blocks;
  if (grid > INT_MAX) return GQA_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (L.dec) {
    s = launch_dec(p, L, di, st);
  } else if (L.tc) {
    if (d == 64)
      s = L.NT == 1 ? launch_tc<64, 1>(p, di, st) : launch_tc<64, 2>(p, di, st);
    else
      s = L.NT == 1 ? launch_tc<128, 1>(p, di, st) : launch_tc<128, 2>(p, di, st);
  } else {
    s = dtype == GQA_F32 ? launch_simt<float>(p, di, st) : launch_simt<__nv_bfloat16>(p, di, st);
  }
  if (s != GQA_OK) return s;
  if (L.finish) {
    auto *kernel = L.part_warps == 4 ? gqa::rows::rows_finish_kernel<__nv_bfloat16, 4>
                                     : gqa::rows::rows_finish_kernel<__nv_bfloat16, 1>;
    s = launched(gqa::launch_dependent(kernel, dim3((unsigned)finish_blocks),
                                       dim3(gqa::rows::kFinishThreads), 0, st, p, row_blocks, col_blocks));
    if (s != GQA_OK) return s;
  }
  if (tree) return s;
  if (!L.scores && L.tc)
    return d == 64 ? launch_weigh_tc<64>(p, di, st) : launch_weigh_tc<128>(p, di, st);
  if (!L.scores)
    return launched(gqa::launch_dependent(
        d == 64 ? gqa::rows::rows_weigh_keys_kernel<64> : gqa::rows::rows_weigh_keys_kernel<128>,
        dim3((unsigned)grid), dim3(gqa::rows::kWeighKeyThreads), 0, st, p, cell_blocks));
  return launched(gqa::launch_dependent(gqa::rows::rows_weigh_kernel, dim3((unsigned)grid),
                                        dim3(gqa::rows::kWeighThreads), 0, st, p, cell_blocks));
}

// The larger of the two layouts: buffers that are not 16-byte aligned run
// the CUDA-core kernel.  (They are of like size: partial sums, and scores where
// either keeps them.)
size_t workspace_bytes_of(gqa_dtype dtype, int B, int Hq, int Hkv, int C, int d, int t, bool scored) {
  if (dtype != GQA_F32 && dtype != GQA_BF16) return 0;
  if (B < 0 || C < 0 || t < 0 || t > GQA_MAX_TREE || check_heads(Hq, Hkv, d) != GQA_OK) return 0;
  if (d > GQA_MAX_HEAD_DIM || C > INT_MAX - 2 * GQA_MAX_TREE) return 0;
  Layout a, b;
  if (!layout(dtype, B, Hq, Hkv, C, d, t, scored, true, &a) ||
      !layout(dtype, B, Hq, Hkv, C, d, t, scored, false, &b))
    return 0;
  return std::max(a.total, b.total);
}

}  // namespace

extern "C" {

size_t gqa_decode_tree_workspace_bytes(gqa_dtype dtype, int B, int Hq, int Hkv, int C, int d,
                                       int t_new) {
  return workspace_bytes_of(dtype, B, Hq, Hkv, C, d, t_new, false);
}

size_t gqa_decode_scored_workspace_bytes(gqa_dtype dtype, int B, int Hq, int Hkv, int C, int d,
                                         int t_new) {
  return workspace_bytes_of(dtype, B, Hq, Hkv, C, d, t_new, true);
}

gqa_status gqa_decode_tree(gqa_dtype dtype, const void *q, const void *k_cache,
                           const void *v_cache, const void *k_draft, const void *v_draft,
                           const int32_t *parents, void *o, const int32_t *seq_lens, int B,
                           int Hq, int Hkv, int C, int d, int t_new, int window, float scale,
                           void *workspace, size_t workspace_bytes, int32_t *dev_status,
                           gqa_stream_t stream) {
  const Operands op{q, k_cache, v_cache, k_draft, v_draft, parents, seq_lens, o, nullptr};
  return rows_impl(dtype, op, true, B, Hq, Hkv, C, d, t_new, window, scale, workspace,
                   workspace_bytes, dev_status, stream);
}

gqa_status gqa_decode_scored(gqa_dtype dtype, const void *q, const void *k_cache,
                             const void *v_cache, void *o, float *weights,
                             const int32_t *seq_lens, int B, int Hq, int Hkv, int C, int d,
                             int t_new, float scale, void *workspace, size_t workspace_bytes,
                             int32_t *dev_status, gqa_stream_t stream) {
  const Operands op{q, k_cache, v_cache, nullptr, nullptr, nullptr, seq_lens, o, weights};
  return rows_impl(dtype, op, false, B, Hq, Hkv, C, d, t_new, GQA_NO_WINDOW, scale, workspace,
                   workspace_bytes, dev_status, stream);
}

}  // extern "C"
