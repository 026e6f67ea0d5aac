// linear_act_backward and gated_ffn_backward: the pass through the activation (and the
// bias gradients), then the two products of the tensor cores.
#include "ffn_host.h"
#include "launch.cuh"

using namespace igc;

namespace {

constexpr size_t kAlign = 256;
size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Row stride of dZ / dG / dU in the workspace.
int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

size_t matrix_bytes(int64_t M, int64_t N) {
  return up(static_cast<size_t>(M) * static_cast<size_t>(padded(N)) * 2);
}
size_t partial_bytes(int64_t M, int64_t N, int vectors) {
  return up(static_cast<size_t>(vectors) * static_cast<size_t>(dact_chunks(M, N)) *
            static_cast<size_t>(N) * 4);
}

// Zeros for a contraction of length zero.
int zero_mat(const Mat& m, int64_t rows, int64_t cols, cudaStream_t stream) {
  return zero_rows(const_cast<void*>(m.ptr), m.ld, rows, cols, elem_size(m.dtype), stream);
}

bool bad_grad_type(const void* p, int t, int dtype) {
  return p != nullptr && t != IGC_F32 && t != dtype;
}

// The part that both operators share, `n` matrices of pre-activations.
int backward(int64_t M, int64_t N, int64_t K, int dtype, int act, bool gated, const Mat& dO,
             const Mat& Z, const Mat& U, const Mat& X, const Mat* W, const Mat& dX, const Mat* dW,
             void* const* db, int db_dtype, void* workspace, size_t workspace_bytes, size_t need,
             cudaStream_t stream) {
  const int n = gated ? 2 : 1;
  const bool want_x = dX.ptr != nullptr && M > 0 && K > 0;
  const bool want_w = dW[0].ptr != nullptr && N > 0 && K > 0;
  const bool want_b = db[0] != nullptr && N > 0;
  if (!want_x && !want_w && !want_b) return IGC_OK;
  // outputs are no inputs and all different
  const void* outs[5] = {dX.ptr, dW[0].ptr, n > 1 ? dW[1].ptr : nullptr, db[0], db[1]};
  for (int i = 0; i < 5; ++i) {
    if (is_any(outs[i], dO.ptr, Z.ptr, U.ptr, X.ptr, W[0].ptr, n > 1 ? W[1].ptr : nullptr))
      return IGC_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (is_any(outs[i], outs[j])) return IGC_ERR_INVALID_ARG;
  }
  if (!fits32(M) || !fits32(N) || !fits32(K)) return IGC_ERR_UNSUPPORTED;
  if (M > 0 && N > 0) {
    if (dO.ptr == nullptr || dO.ld < N) return IGC_ERR_INVALID_ARG;
    if ((gated || act != IGC_ACT_NONE) && (Z.ptr == nullptr || Z.ld < N))
      return IGC_ERR_INVALID_ARG;
    if (gated && U.ptr == nullptr) return IGC_ERR_INVALID_ARG;
    if (want_w && (X.ptr == nullptr || X.ld < K)) return IGC_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
      if (want_x && (W[i].ptr == nullptr || W[i].ld < K)) return IGC_ERR_INVALID_ARG;
    if (want_w && !operand_ok(X.ptr, X.ld)) return IGC_ERR_MISALIGNED;
    for (int i = 0; i < n; ++i)
      if (want_x && !operand_ok(W[i].ptr, W[i].ld)) return IGC_ERR_MISALIGNED;
    if (!elements_aligned(dO, U) || ((gated || act != IGC_ACT_NONE) && !elements_aligned(Z)))
      return IGC_ERR_MISALIGNED;
  }
  if ((want_x && !elements_aligned(dX)) ||
      (want_b && !elements_aligned(Mat{db[0], N, db_dtype}, Mat{db[1], N, db_dtype})))
    return IGC_ERR_MISALIGNED;
  for (int i = 0; i < n; ++i)
    if (want_w && !elements_aligned(dW[i])) return IGC_ERR_MISALIGNED;

  DeviceInfo dev;
  int rc = current_device(&dev);
  if (rc != IGC_OK) return rc;

  if (M == 0 || N == 0) {  // empty sums
    if (want_x) rc = zero_mat(dX, M, K, stream);
    for (int i = 0; i < n && rc == IGC_OK; ++i) {
      if (want_w) rc = zero_mat(dW[i], N, K, stream);
      if (rc == IGC_OK && want_b) rc = zero_mat({db[i], N, db_dtype}, 1, N, stream);
    }
    return rc;
  }

  // Without an activation dZ is dY itself; it is copied only when TMA cannot read it.
  const bool identity = !gated && act == IGC_ACT_NONE;
  const bool copy = (want_x || want_w) && (!identity || !operand_ok(dO.ptr, dO.ld));
  Mat D[2] = {{dO.ptr, dO.ld, dtype}, {}};
  // Plans of both products, whether or not both are asked for, so that a gradient does not
  // depend on that.
  GradArgs g;
  g.M = M, g.N = N, g.K = K, g.dtype = dtype, g.count = n;
  g.D = D, g.W = W, g.X = X, g.dX = dX, g.dW = dW;
  ProductPlan px, pw;
  if (want_x || want_w) {
    rc = ffn_plan_x(dev, g, &px);
    if (rc == IGC_OK) rc = ffn_plan_w(dev, g, &pw);
    if (rc != IGC_OK) return rc;
    if (grad_x_beside_w(px, pw, dev.sm_count)) px.small = false;
  }

  DactArgs a;
  if (copy || want_b) {
    if (workspace == nullptr || workspace_bytes < need ||
        reinterpret_cast<uintptr_t>(workspace) % kAlign != 0)
      return IGC_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.M = M, a.N = N, a.dtype = dtype, a.act = act;
    a.dO = dO, a.Z = Z, a.U = U;
    a.ldd = padded(N);
    if (copy) {
      for (int i = 0; i < n; ++i) D[i] = {ws + i * matrix_bytes(M, N), padded(N), dtype};
      a.D0 = const_cast<void*>(D[0].ptr);
      a.D1 = const_cast<void*>(D[1].ptr);
    }
    if (want_b) {
      a.db0 = db[0], a.db1 = db[1], a.db_dtype = db_dtype;
      a.partial = reinterpret_cast<float*>(ws + n * matrix_bytes(M, N));
    }
    rc = ffn_dact(a, gated, stream);
    if (rc != IGC_OK) return rc;
  }
  // What follows reads what the activation's pass wrote and nothing of one another: each
  // kernel but the first may run beside those before it (late_wait, ffn_dependency_wait).
  bool after_first = false;
  if (want_x) {
    rc = ffn_grad_x(dev, g, px, after_first, stream);
    if (rc != IGC_OK) return rc;
    after_first = true;
  }
  if (want_w) {
    rc = ffn_grad_w(dev, g, pw, after_first, stream);
    if (rc != IGC_OK) return rc;
    after_first = true;
  }
  if (want_b) rc = ffn_dact_sums(a, gated, after_first, stream);
  return rc;
}

}  // namespace

extern "C" {

size_t linear_act_backward_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return 0;
  return matrix_bytes(M, N) + partial_bytes(M, N, 1);
}

int linear_act_backward(int64_t M, int64_t N, int64_t K, int dtype, const void* dY, int64_t lddy,
                        const void* Z, int64_t ldz, int act, const void* X, int64_t ldx,
                        const void* W, int64_t ldw, void* dX, int64_t lddx, void* dW,
                        int64_t lddw, int dw_dtype, void* dbias, int dbias_dtype,
                        void* workspace, size_t workspace_bytes, igc_stream_t stream) {
  if (M < 0 || N < 0 || K < 0 || !is_operand_type(dtype)) return IGC_ERR_INVALID_ARG;
  if (act < IGC_ACT_NONE || act > IGC_ACT_SILU) return IGC_ERR_INVALID_ARG;
  if (bad_grad_type(dW, dw_dtype, dtype) || bad_grad_type(dbias, dbias_dtype, dtype))
    return IGC_ERR_INVALID_ARG;
  if ((dX != nullptr && lddx < K) || (dW != nullptr && lddw < K)) return IGC_ERR_INVALID_ARG;
  const Mat w{W, ldw, dtype}, dw{dW, lddw, dw_dtype};
  void* db[2] = {dbias, nullptr};
  return backward(M, N, K, dtype, act, false, {dY, lddy, dtype}, {Z, ldz, dtype}, {},
                  {X, ldx, dtype}, &w, {dX, lddx, dtype}, &dw, db, dbias_dtype, workspace,
                  workspace_bytes, linear_act_backward_workspace_size(M, N, K),
                  reinterpret_cast<cudaStream_t>(stream));
}

size_t gated_ffn_backward_workspace_size(int64_t M, int64_t F, int64_t K) {
  if (M < 0 || F < 0 || K < 0) return 0;
  return 2 * matrix_bytes(M, F) + partial_bytes(M, F, 2);
}

int gated_ffn_backward(int64_t M, int64_t F, int64_t K, int dtype, const void* dH, int64_t lddh,
                       const void* G, const void* U, int64_t ldgu, int act, const void* X,
                       int64_t ldx, const void* Wg, const void* Wu, int64_t ldw, void* dX,
                       int64_t lddx, void* dWg, void* dWu, int64_t lddw, int dw_dtype, void* dbg,
                       void* dbu, int dbias_dtype, void* workspace, size_t workspace_bytes,
                       igc_stream_t stream) {
  if (M < 0 || F < 0 || K < 0 || !is_operand_type(dtype)) return IGC_ERR_INVALID_ARG;
  if (act < IGC_ACT_NONE || act > IGC_ACT_SILU) return IGC_ERR_INVALID_ARG;
  if ((dWg == nullptr) != (dWu == nullptr) || (dbg == nullptr) != (dbu == nullptr))
    return IGC_ERR_INVALID_ARG;
  if (bad_grad_type(dWg, dw_dtype, dtype) || bad_grad_type(dbg, dbias_dtype, dtype))
    return IGC_ERR_INVALID_ARG;
  if ((dX != nullptr && lddx < K) || (dWg != nullptr && lddw < K)) return IGC_ERR_INVALID_ARG;
  const Mat w[2] = {{Wg, ldw, dtype}, {Wu, ldw, dtype}};
  const Mat dw[2] = {{dWg, lddw, dw_dtype}, {dWu, lddw, dw_dtype}};
  void* db[2] = {dbg, dbu};
  return backward(M, F, K, dtype, act, true, {dH, lddh, dtype}, {G, ldgu, dtype},
                  {U, ldgu, dtype}, {X, ldx, dtype}, w, {dX, lddx, dtype}, dw, db, dbias_dtype,
                  workspace, workspace_bytes, gated_ffn_backward_workspace_size(M, F, K),
                  reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
