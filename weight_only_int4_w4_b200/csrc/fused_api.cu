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

size_t fused_ws_bytes(int64_t M, int64_t N, int64_t K, bool gated, bool grad) {
  (void)K;
  (void)gated;
  return grad ? kCounterBytes + (size_t)M * N * 4 : 0;
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
  for (const Buf &o : outs)
    for (const Buf &i : ins)
      if (overlap(o.p, o.n, i.p, i.n) && !(i.p == c.residual && o.p == c.Y && c.residual == c.Y))
        return fail(W4_ERR_INVALID_ARG, "an output overlaps an input or the workspace");
  for (int a = 0; a < 3; ++a)
    for (int b = a + 1; b < 3; ++b)
      if (overlap(outs[a].p, outs[a].n, outs[b].p, outs[b].n))
        return fail(W4_ERR_INVALID_ARG, "two outputs overlap");
  for (int i = 0; i < 8; ++i)
    if (overlap(c.workspace, c.workspace_bytes, ins[i].p, ins[i].n))
      return fail(W4_ERR_INVALID_ARG, "the workspace overlaps an input");
  const size_t need = fused_ws_bytes(c.M, c.N, c.K, c.gated, c.grad);
  if (need > 0 && (!c.workspace || c.workspace_bytes < need))
    return fail(W4_ERR_INVALID_ARG, "workspace too small: need %zu bytes, got %zu", need,
                c.workspace ? c.workspace_bytes : (size_t)0);
  return W4_OK;
}

w4_status fused_run(const FusedCall &c, w4_stream_t stream) {
  t_last_error.clear();
  const w4_status st = fused_check(c);
  if (st != W4_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  w4::FusedParams p{};
  p.X = c.X; p.x_dtype = (int)c.x_dtype;
  p.M = c.M; p.N = c.N; p.K = c.K; p.group = c.group;
  p.packed = c.packed; p.scales = c.scales; p.zeros = c.zeros; p.awq_s = c.awq_s; p.bias = c.bias;
  p.act = (int)c.act; p.residual = c.residual; p.Z = c.Z; p.Y = c.Y; p.y_dtype = (int)c.y_dtype;
  cudaError_t e;
  if (!c.grad) e = w4::launch_fused_simple(p, c.gated, s);
  else
    e = w4::launch_fused_grad_simple(p, c.gated, c.X, c.Z,
                                     reinterpret_cast<float *>(static_cast<uint8_t *>(c.workspace) + kCounterBytes),
                                     c.dbias, s);
  if (e != cudaSuccess) return cuda_fail(e, "fused operator launch");
  return W4_OK;
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
