// fused_api.cu -- host side of the fused operators (included by libw4.cu): argument
// checks before anything is launched, workspace layout, launch.

namespace {

struct FusedCall {
  const void *X;  // X, or dY / dH
  w4_dtype x_dtype;
  int64_t M, N, K;  // N: packed rows (2F for gated)
  int group;
  const uint8_t *packed;
  const uint16_t *scales, *zeros;
  const float *awq_s, *bias;
  w4_act act;
  const void *residual;
  void *Z, *Y;  // Y: Y, H or dX
  w4_dtype y_dtype;
  float *dbias;
  void *workspace;
  size_t workspace_bytes;
  bool gated, grad;
};

bool overlap(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Rows of a gated layer's packed matrix; sizes that 2F would overflow stay invalid (0).
int64_t gated_rows(int64_t F) { return F < 1 || F > INT32_MAX / 2 ? 0 : 2 * F; }

size_t dtype_size(w4_dtype t) { return t == W4_F32 ? 4 : 2; }

// Launch plan and workspace of a fused call.
struct FusedPlan {
  int bn = 16, mt = 1, rt = 1, units = 1, gt = 1, full = 0, tiles = 1, tail_pairs = 0, pairs = 1;
  int64_t ld = 0;  // row stride of the staged operand
  size_t xp = 0, tinv = 0, rinv = 0, tab = 0, part = 0, dbias = 0, bytes = 0;
};

// Fragments of a cut tile hold at least this many 128-deep units.
constexpr int64_t kMinTailUnits = 2;

// sizes whose tiles or blocks would not fit a grid are refused (false)
bool fused_plan(int64_t M, int64_t N, int64_t K, bool gated, bool grad, int sm, FusedPlan &p) {
  const int64_t rows = grad ? K : gated ? N / 2 : N, depth = grad ? N : K;
  const int64_t mt = cdiv(M, w4::ftc::kMaxBn), rt = cdiv(rows, gated && !grad ? 128 : 256), units = cdiv(depth, 128);
  const int pairs = sm / 2;
  if (M > (int64_t)1 << 30 || (double)rt * (double)mt > 1.0e9) return false;
  p.mt = (int)mt;
  p.bn = (int)(cdiv(cdiv(M, mt), 32) * 32);
  p.rt = (int)rt;
  p.units = (int)units;
  p.gt = (int)std::min<int64_t>(mt, 8);
  p.tiles = (int)(rt * mt);
  p.full = p.tiles / pairs * pairs;
  const int64_t rest = p.tiles - p.full;
  if (rest > 0) {
    const int64_t share = std::min<int64_t>(pairs, rest * units / kMinTailUnits);
    if (share > rest && rest * 10 < 9 * (int64_t)pairs) p.tail_pairs = (int)share;
    else p.full = p.tiles;
  }
  p.pairs = p.full > 0 ? std::min(pairs, std::max(p.full, p.tail_pairs)) : p.tail_pairs;
  p.ld = grad ? cdiv(N, 8) * 8 : K;
  p.xp = kCounterBytes;
  p.tinv = p.xp + align256((size_t)M * p.ld * 2);
  p.rinv = p.tinv + align256((size_t)M * 4);
  p.tab = p.rinv + align256((size_t)N * 4);
  p.part = p.tab + align256((size_t)N * (K / 32) * 4);  // room for groups of 32
  p.dbias = p.part + align256((size_t)4 * p.tail_pairs * p.bn * 128 * 4);
  const size_t db = !grad ? 0 : (size_t)w4::fused_dbias_parts(M, N, gated, sm) * N * 4;
  p.bytes = p.dbias + align256(db);
  return true;
}

// Up to 8 tokens on groups of 128: one kernel, no workspace.  Splits K over as many of a
// CTA's 16 warps as there are pieces of channels and room for the partial sums; ranges of
// rows are as many as SMs (or clusters), or a multiple where the partial sums of one would
// not fit.  Clusters of 2 or 4 where a CTA's activations would be over a quarter of its
// weights (2 M K bytes against N K / 2 / SMs).
struct GemvFusedPlan {
  int grid = 0, ksw = 1, nblk = 1, cluster = 1, depth = 3;
};
bool fused_gemv_plan(int64_t M, int64_t N, int64_t K, int group, bool gated, int sm, GemvFusedPlan &p) {
  if (group != w4::kGroup || M > w4::fgv::kMaxTokens) return false;
  if ((double)N * (double)(K / w4::kGroup) > 4.0e9) return false;  // groups are numbered in 32 bits
  const int64_t out = gated ? N / 2 : N, pieces = cdiv(K / w4::kGroup, 2);
  int cluster = 1;
  while (cluster < 4 && 2.0 * M / cluster > 0.125 * (double)N / sm && pieces >= 4 * cluster) cluster *= 2;
  const int64_t most = w4::fused_gemv_clusters(cluster, sm);
  for (int64_t ranges = std::min<int64_t>(most, cdiv(out, 8)); ranges <= (int64_t)1 << 20; ranges *= 2) {
    const int64_t nblk = cdiv(cdiv(out, ranges), 16) * (gated ? 2 : 1);
    for (int ksw = 16; ksw >= 1; ksw /= 2)
      for (int depth = 4; depth >= 3; --depth) {
        if (ksw * cluster > pieces ||
            w4::fgv::smem_bytes(ksw, (int)std::min<int64_t>(nblk, 1 << 16), (int)M, cluster, depth) > w4::fgv::kSmemMax)
          continue;
        p.grid = (int)ranges * cluster;
        p.ksw = ksw;
        p.nblk = (int)nblk;
        p.cluster = cluster;
        p.depth = depth;
        return true;
      }
  }
  return false;
}

// 9 to 64 tokens on groups of 128, on the tensor cores.  For 1, 2, 4 or 8 CTAs to a range of
// rows, the cycles of a CTA: its (tile, group) pairs, each the larger of what the bytes of
// a tile's rows take at an SM's share of HBM and what their conversion takes.
struct SkinnyFusedPlan {
  int grid = 0, cluster = 1, tiles = 1, tile_rows = 0, bn = 16;
  size_t xp = 0, tinv = 0, bytes = 0;
};
bool fused_skinny_plan(int64_t M, int64_t N, int64_t K, int group, bool gated, int sm, SkinnyFusedPlan &p) {
  if (group != w4::kGroup || K % w4::kGroup != 0 || M > w4::fsk::kMaxTokens) return false;
  constexpr double kConvert = 300.0, kBytesPerCycle = 23.4, kCluster = 2000.0;
  const int64_t out = gated ? N / 2 : N, Kg = K / w4::kGroup, lim = gated ? 64 : 128;
  p.bn = (int)(cdiv(M, 16) * 16);
  double best = 0;
  for (int cluster = 1; cluster <= 8 && cluster <= Kg; cluster *= 2) {
    const int64_t ranges = std::min<int64_t>(w4::fused_gemv_clusters(cluster, sm), cdiv(out, 8));
    const int64_t rows = cdiv(out, ranges), tiles = cdiv(rows, lim), tile_rows = cdiv(rows, tiles);
    if (tiles > 1 << 20 || tiles * cdiv(Kg, cluster) > 1 << 30 ||
        w4::fsk::code_stages(p.bn, (int)M, (int)std::min<int64_t>(tiles, 512), cluster) < w4::fsk::kMinCodeStages)
      continue;
    const double unit = std::max(kConvert, (double)tile_rows * (gated ? 2 : 1) * 68.0 / kBytesPerCycle);
    const double cost = (double)tiles * (double)cdiv(Kg, cluster) * unit + (cluster > 1 ? kCluster : 0.0);
    if (p.grid == 0 || cost < best) {
      best = cost;
      p.grid = (int)ranges * cluster;
      p.cluster = cluster;
      p.tiles = (int)tiles;
      p.tile_rows = (int)tile_rows;
    }
  }
  p.xp = kCounterBytes;
  p.tinv = p.xp + align256((size_t)K * p.bn * 2);
  p.bytes = p.tinv + align256((size_t)p.bn * 4);
  return p.grid > 0;
}

int sm_count_or_b200() {
  int sm = 0;
  return current_sm_count(&sm) == cudaSuccess ? sm : 148;
}

size_t fused_ws_bytes(int64_t M, int64_t N, int64_t K, bool gated, bool grad) {
  FusedPlan p;
  const int sm = sm_count_or_b200();
  if (!fused_plan(M, N, K, gated, grad, sm, p)) return 0;
  SkinnyFusedPlan sp;
  if (!grad && fused_skinny_plan(M, N, K, w4::kGroup, gated, sm, sp)) return std::max(p.bytes, sp.bytes);
  return p.bytes;
}

// Which kernel serves a call.  Measured on B200 at the 8B and 70B layer shapes, microseconds of
// decode / small-batch kernel: 8 tokens 9.4 / 12 (4096 x 4096), 19 / 23 (14336 -> 4096), 25 /
// 30 (4096 -> 2 x 14336), 72 / 97 (8192 -> 2 x 28672); 16 tokens 14 / 12, 28 / 23, 43 / 30,
// 128 / 97.  Small-batch / prefill kernel at 64 tokens: 15 / 25, 27 / 41, 36 / 51, 110 / 140.
enum FusedRoute { kRouteDecode, kRouteSkinny, kRouteTc };
FusedRoute fused_route(const FusedCall &c) {
  if (c.grad || c.group != w4::kGroup || c.M > w4::fsk::kMaxTokens) return kRouteTc;
  return c.M <= w4::fgv::kMaxTokens ? kRouteDecode : kRouteSkinny;
}

// Everything a fused call can be refused for, checked on the host.
w4_status fused_check(const FusedCall &c) {
  w4_status st = check_shape(c.M, c.N, c.K, c.group);
  if (st != W4_OK) return st;
  if (c.K % 64 != 0) return fail(W4_ERR_UNSUPPORTED, "K=%lld must be a multiple of 64", (long long)c.K);
  if (c.x_dtype != W4_F16 && c.x_dtype != W4_BF16)
    return fail(W4_ERR_UNSUPPORTED, "%s dtype must be F16 or BF16", c.grad ? "gradient" : "activation");
  if (c.y_dtype != W4_F32 && c.y_dtype != W4_F16 && c.y_dtype != W4_BF16)
    return fail(W4_ERR_UNSUPPORTED, "output dtype %d not served", (int)c.y_dtype);
  if (c.act < W4_ACT_NONE || c.act > W4_ACT_GELU_TANH)
    return fail(W4_ERR_UNSUPPORTED, "activation %d not served", (int)c.act);
  if (!c.X || !c.packed || !c.scales || !c.zeros || !c.Y)
    return fail(W4_ERR_INVALID_ARG, "null %s, packed, scales, zeros or output", c.grad ? "gradient" : "X");
  if (c.grad && (c.gated || c.act != W4_ACT_NONE) && !c.Z)
    return fail(W4_ERR_INVALID_ARG, "the gradient of an activated product needs its pre-activations");
  const void *ptrs[] = {c.X, c.packed, c.scales, c.zeros, c.awq_s, c.bias, c.residual, c.Z, c.Y, c.dbias, c.workspace};
  for (const void *p : ptrs)
    if (!aligned16(p)) return fail(W4_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
  // Outputs may not overlap what the call still reads.  Y may be the residual itself
  // (each element is read and then written by one thread).
  const int64_t out = c.gated ? c.N / 2 : c.N;
  const size_t xb = (size_t)c.M * (c.grad ? out : c.K) * 2;
  const size_t yb = (size_t)c.M * (c.grad ? c.K : out) * dtype_size(c.y_dtype);
  const size_t zb = (size_t)c.M * c.N * 2, rb = (size_t)c.M * c.N * dtype_size(c.y_dtype);
  const size_t pb = (size_t)c.N * (size_t)(c.K / 2), sb = (size_t)c.N * (size_t)(c.K / c.group) * 2;
  const size_t kb = (size_t)c.K * 4, nb = (size_t)c.N * 4;
  struct Buf { const void *p; size_t n; };
  const Buf ins[] = {{c.X, xb}, {c.packed, pb}, {c.scales, sb}, {c.zeros, sb}, {c.awq_s, kb}, {c.bias, nb},
                     {c.residual, rb}, {c.grad ? c.Z : nullptr, zb}, {c.workspace, c.workspace_bytes}};
  const Buf outs[] = {{c.Y, yb}, {c.grad ? nullptr : c.Z, zb}, {c.dbias, nb}};
  constexpr int kResidual = 6;  // its place in ins; by address, another input that lies there too would pass
  for (const Buf &o : outs)
    for (int i = 0; i < 9; ++i)
      if (overlap(o.p, o.n, ins[i].p, ins[i].n) && !(i == kResidual && o.p == c.Y && c.residual == c.Y))
        return fail(W4_ERR_INVALID_ARG, "an output overlaps an input or the workspace");
  for (int a = 0; a < 3; ++a)
    for (int b = a + 1; b < 3; ++b)
      if (overlap(outs[a].p, outs[a].n, outs[b].p, outs[b].n))
        return fail(W4_ERR_INVALID_ARG, "two outputs overlap");
  for (int i = 0; i < 8; ++i)
    if (overlap(c.workspace, c.workspace_bytes, ins[i].p, ins[i].n))
      return fail(W4_ERR_INVALID_ARG, "the workspace overlaps an input");
  if (fused_route(c) == kRouteDecode) return W4_OK;  // takes no workspace
  const size_t need = fused_ws_bytes(c.M, c.N, c.K, c.gated, c.grad);
  if (need == 0)
    return fail(W4_ERR_INVALID_ARG, "M=%lld N=%lld K=%lld: too many tiles for one launch", (long long)c.M, (long long)c.N,
                (long long)c.K);
  if (!c.workspace || c.workspace_bytes < need)
    return fail(W4_ERR_INVALID_ARG, "workspace too small: need %zu bytes, got %zu", need,
                c.workspace ? c.workspace_bytes : (size_t)0);
  return W4_OK;
}

// The tensor-core path: operand staging, the product, and the sum of cut tiles.
w4_status fused_run_tc(const FusedCall &c, const FusedPlan &plan, int sm, cudaStream_t s) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  uint8_t *ws = static_cast<uint8_t *>(c.workspace);
  uint16_t *xp = reinterpret_cast<uint16_t *>(ws + plan.xp);
  float *tinv = reinterpret_cast<float *>(ws + plan.tinv), *rinv = reinterpret_cast<float *>(ws + plan.rinv);
  uint32_t *tab = reinterpret_cast<uint32_t *>(ws + plan.tab);
  const int64_t kg = c.K / c.group, depth = c.grad ? plan.ld : c.K;
  CUtensorMap tmX, tmP;
  CUresult r = encode_2d(enc, &tmX, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xp, (uint64_t)depth, (uint64_t)c.M,
                         (uint64_t)plan.ld * 2, 64u, (uint32_t)plan.bn / 2, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r != CUDA_SUCCESS) return fail(W4_ERR_CUDA, "tensor map for staged operands failed (CUresult %d)", (int)r);
  r = encode_2d(enc, &tmP, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.packed, (uint64_t)(c.K / 2), (uint64_t)c.N,
                (uint64_t)(c.K / 2), 64u, c.gated && !c.grad ? 64u : 128u, CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r != CUDA_SUCCESS) return fail(W4_ERR_CUDA, "tensor map for packed weights failed (CUresult %d)", (int)r);
  cudaError_t e;
  int64_t sums = 0;  // rows of dbias's partial sums that are still to be added
  if (c.grad) {
    e = w4::launch_fused_stage_dz(c.X, c.act == W4_ACT_NONE && !c.gated ? nullptr : c.Z, (int)c.x_dtype, (int)c.act,
                                  c.gated, c.M, c.N, plan.ld, c.scales, c.zeros, kg, xp, tinv, rinv, tab,
                                  reinterpret_cast<float *>(ws + plan.dbias), c.dbias, sm, &sums, s);
  } else {
    e = w4::launch_fused_stage_x(c.X, c.x_dtype == W4_BF16, c.awq_s, c.M, c.K, c.scales, c.zeros, kg, c.N, xp, tinv, rinv,
                                 tab, s);
  }
  if (e != cudaSuccess) return cuda_fail(e, "operand staging launch");
  w4::FusedTcParams p{};
  p.epi.M = c.M;
  p.epi.N = c.grad ? c.K : c.gated ? c.N / 2 : c.N;
  p.epi.rinv = rinv; p.epi.tinv = tinv;
  p.epi.bias = c.bias;
  p.epi.colmul = c.grad ? c.awq_s : nullptr;
  p.epi.residual = c.residual; p.epi.Z = c.grad ? nullptr : c.Z; p.epi.Y = c.Y;
  p.epi.act = c.grad ? (int)W4_ACT_NONE : (int)c.act;
  p.epi.z_dtype = (int)c.x_dtype; p.epi.y_dtype = (int)c.y_dtype;
  p.epi.vec = p.epi.N % 4 == 0;
  p.tab = tab;
  p.rows = c.N; p.kg = kg;
  p.gshift = c.group == 128 ? 7 : c.group == 64 ? 6 : 5;
  p.bn = plan.bn; p.mt = plan.mt; p.rt = plan.rt; p.units = plan.units; p.gt = plan.gt;
  p.full = plan.full; p.tiles = plan.tiles; p.tail_pairs = plan.tail_pairs;
  p.part = reinterpret_cast<float *>(ws + plan.part);
  e = w4::launch_fused_tc(c.grad ? w4::kGrad : c.gated ? w4::kGated : w4::kLinear, tmX, tmP, p, plan.pairs, s);
  if (e != cudaSuccess) return cuda_fail(e, "fused product launch");
  if (c.dbias) {
    e = w4::launch_fused_dbias_sum(c.N, sums, reinterpret_cast<const float *>(ws + plan.dbias), c.dbias, s);
    if (e != cudaSuccess) return cuda_fail(e, "bias gradient launch");
  }
  return W4_OK;
}

w4_status fused_run_skinny(const FusedCall &c, const SkinnyFusedPlan &plan, cudaStream_t s) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  uint8_t *ws = static_cast<uint8_t *>(c.workspace);
  uint16_t *xp = reinterpret_cast<uint16_t *>(ws + plan.xp);
  float *tinv = reinterpret_cast<float *>(ws + plan.tinv);
  CUtensorMap tmX, tmP;
  CUresult r = encode_2d(enc, &tmX, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, xp, 64u, (uint64_t)(c.K / 64) * plan.bn, 128u, 64u,
                         2u * plan.bn, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r != CUDA_SUCCESS) return fail(W4_ERR_CUDA, "tensor map for staged activations failed (CUresult %d)", (int)r);
  r = encode_2d(enc, &tmP, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.packed, (uint64_t)(c.K / 2), (uint64_t)c.N,
                (uint64_t)(c.K / 2), 128u, (uint32_t)plan.tile_rows, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r != CUDA_SUCCESS) return fail(W4_ERR_CUDA, "tensor map for packed weights failed (CUresult %d)", (int)r);
  cudaError_t e = w4::launch_fused_stage_small(c.X, c.x_dtype == W4_BF16, c.awq_s, c.M, c.K, plan.bn, xp, tinv, s);
  if (e != cudaSuccess) return cuda_fail(e, "activation staging launch");
  w4::FusedSkinnyParams p{};
  p.epi.M = c.M; p.epi.N = c.gated ? c.N / 2 : c.N;
  p.epi.tinv = tinv; p.epi.bias = c.bias; p.epi.residual = c.residual; p.epi.Z = c.Z; p.epi.Y = c.Y;
  p.epi.act = (int)c.act; p.epi.z_dtype = (int)c.x_dtype; p.epi.y_dtype = (int)c.y_dtype;
  p.scales = c.scales; p.zeros = c.zeros;
  p.groups = (int)(c.K / w4::kGroup);
  p.tile_rows = plan.tile_rows; p.tiles = plan.tiles; p.cluster = plan.cluster;
  p.code_stages = w4::fsk::code_stages(plan.bn, (int)c.M, plan.tiles, plan.cluster);
  e = w4::launch_fused_skinny(tmX, tmP, p, c.gated, plan.grid, s);
  if (e != cudaSuccess) return cuda_fail(e, "fused small-batch launch");
  return W4_OK;
}

w4_status fused_run_gemv(const FusedCall &c, const GemvFusedPlan &plan, cudaStream_t s) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return fail(W4_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  CUtensorMap tmP;
  const CUresult r = encode_2d(enc, &tmP, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.packed, (uint64_t)(c.K / 2), (uint64_t)c.N,
                               (uint64_t)(c.K / 2), 128u, 16u, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (r != CUDA_SUCCESS) return fail(W4_ERR_CUDA, "tensor map for packed weights failed (CUresult %d)", (int)r);
  w4::FusedGemvParams p{};
  p.X = static_cast<const uint16_t *>(c.X);
  p.M = c.M; p.N = c.gated ? c.N / 2 : c.N; p.K = c.K;
  p.scales = c.scales; p.zeros = c.zeros; p.awq_s = c.awq_s;
  p.epi.bias = c.bias; p.epi.residual = c.residual; p.epi.Z = c.Z; p.epi.Y = c.Y;
  p.epi.act = (int)c.act; p.epi.z_dtype = (int)c.x_dtype; p.epi.y_dtype = (int)c.y_dtype;
  p.depth = plan.depth;
  p.ksw = plan.ksw; p.nblk = plan.nblk; p.cluster = plan.cluster;
  const cudaError_t e = w4::launch_fused_gemv(tmP, p, c.gated, c.x_dtype == W4_BF16, plan.grid, s);
  if (e != cudaSuccess) return cuda_fail(e, "fused decode launch");
  return W4_OK;
}

w4_status fused_run(const FusedCall &c, w4_stream_t stream) {
  t_last_error.clear();
  const w4_status st = fused_check(c);
  if (st != W4_OK) return st;
  int sm = 0;
  cudaError_t e = current_sm_count(&sm);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  const FusedRoute route = fused_route(c);
  if (route == kRouteDecode) {
    GemvFusedPlan gv;
    if (!fused_gemv_plan(c.M, c.N, c.K, c.group, c.gated, sm, gv))
      return fail(W4_ERR_INVALID_ARG, "N=%lld K=%lld: too many groups for one launch", (long long)c.N, (long long)c.K);
    return fused_run_gemv(c, gv, reinterpret_cast<cudaStream_t>(stream));
  }
  SkinnyFusedPlan sk;
  // (not where the tiles of a range pass what one CTA counts: the prefill kernel then)
  if (route == kRouteSkinny && fused_skinny_plan(c.M, c.N, c.K, c.group, c.gated, sm, sk))
    return fused_run_skinny(c, sk, reinterpret_cast<cudaStream_t>(stream));
  FusedPlan plan;
  fused_plan(c.M, c.N, c.K, c.gated, c.grad, sm, plan);
  return fused_run_tc(c, plan, sm, reinterpret_cast<cudaStream_t>(stream));
}

size_t fused_ws_query(int64_t M, int64_t N, int64_t K, bool gated, bool grad) {
  if (M < 1 || N < 1 || K < 1 || K % 64 != 0) return 0;
  return fused_ws_bytes(M, N, K, gated, grad);
}

}  // namespace

extern "C" {

w4_status w4a16_linear(const void *X, w4_dtype x_dtype, int64_t M, int64_t N, int64_t K, int group,
                       const uint8_t *packed, const uint16_t *scales, const uint16_t *zeros, const float *awq_s,
                       const float *bias, w4_act act, const void *residual, void *Z, void *Y, w4_dtype y_dtype,
                       void *workspace, size_t workspace_bytes, w4_stream_t stream) {
  return fused_run({X, x_dtype, M, N, K, group, packed, scales, zeros, awq_s, bias, act, residual, Z, Y, y_dtype,
                    nullptr, workspace, workspace_bytes, false, false}, stream);
}

w4_status w4a16_gated(const void *X, w4_dtype x_dtype, int64_t M, int64_t F, int64_t K, int group,
                      const uint8_t *packed, const uint16_t *scales, const uint16_t *zeros, const float *awq_s,
                      const float *bias, w4_act act, void *Z, void *H, w4_dtype h_dtype, void *workspace,
                      size_t workspace_bytes, w4_stream_t stream) {
  return fused_run({X, x_dtype, M, gated_rows(F), K, group, packed, scales, zeros, awq_s, bias, act, nullptr, Z, H,
                    h_dtype, nullptr, workspace, workspace_bytes, true, false}, stream);
}

w4_status w4a16_linear_grad(const void *dY, w4_dtype dy_dtype, int64_t M, int64_t N, int64_t K, int group,
                            const uint8_t *packed, const uint16_t *scales, const uint16_t *zeros, const float *awq_s,
                            const void *Z, w4_act act, void *dX, w4_dtype dx_dtype, float *dbias, void *workspace,
                            size_t workspace_bytes, w4_stream_t stream) {
  return fused_run({dY, dy_dtype, M, N, K, group, packed, scales, zeros, awq_s, nullptr, act, nullptr,
                    const_cast<void *>(Z), dX, dx_dtype, dbias, workspace, workspace_bytes, false, true}, stream);
}

w4_status w4a16_gated_grad(const void *dH, w4_dtype dh_dtype, int64_t M, int64_t F, int64_t K, int group,
                           const uint8_t *packed, const uint16_t *scales, const uint16_t *zeros, const float *awq_s,
                           const void *Z, w4_act act, void *dX, w4_dtype dx_dtype, float *dbias, void *workspace,
                           size_t workspace_bytes, w4_stream_t stream) {
  return fused_run({dH, dh_dtype, M, gated_rows(F), K, group, packed, scales, zeros, awq_s, nullptr, act, nullptr,
                    const_cast<void *>(Z), dX, dx_dtype, dbias, workspace, workspace_bytes, true, true}, stream);
}

size_t w4a16_linear_workspace_size(int64_t M, int64_t N, int64_t K) { return fused_ws_query(M, N, K, false, false); }
size_t w4a16_gated_workspace_size(int64_t M, int64_t F, int64_t K) {
  return fused_ws_query(M, gated_rows(F), K, true, false);
}
size_t w4a16_linear_grad_workspace_size(int64_t M, int64_t N, int64_t K) {
  return fused_ws_query(M, N, K, false, true);
}
size_t w4a16_gated_grad_workspace_size(int64_t M, int64_t F, int64_t K) {
  return fused_ws_query(M, gated_rows(F), K, true, true);
}

}  // extern "C"
