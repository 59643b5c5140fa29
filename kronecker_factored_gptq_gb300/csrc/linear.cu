// Entry points of the quantised linear layer: argument checks and the choice
// of kernel.
#include <algorithm>

#include "linear.cuh"

namespace bakron {
namespace {

// Arguments both directions share; T = 0 is a valid call that does nothing.
bool linear_args(const void* x, int64_t T, int dtype, const bakron_packed* w, const void* y,
                 LinearArgs* a) {
  if (!dtype_ok(dtype) || T < 0 || T > (int64_t(1) << 28) || !packed_view(w, &a->w)) return false;
  if (a->w.count != 1) return false;
  if (T > 0 && (!x || !y || !aligned_to(x, dtype_size(dtype)) || !aligned_to(y, dtype_size(dtype))))
    return false;
  a->x = x;
  a->y = const_cast<void*>(y);
  a->T = T;
  a->dtype = dtype;
  return true;
}

size_t workspace_bytes(const LinearArgs& a, bool grad) {
  if (!grad && a.T <= kFewTokens) return 0;
  return linear_tc_workspace(a.T, grad ? a.w.m : a.w.n, a.dtype);
}

bakron_status run_linear(LinearArgs& a, bool grad, void* ws, size_t ws_bytes, void* stream) {
  if (a.T == 0) return BAKRON_OK;
  const size_t need = workspace_bytes(a, grad);
  if (need > 0 && (!ws || !aligned_to(ws, 256) || ws_bytes < need)) return BAKRON_ERR_INVALID_ARG;
  a.ws = ws;
  cudaStream_t s = (cudaStream_t)stream;
  if (!grad && a.T <= kFewTokens)
    return launch_status(launch_linear_few(a, s));
  if (!grad && a.T <= kMidTokens && a.dtype != BAKRON_F32) return launch_status(launch_linear_mid(a, s));
  if (!prop_tc_supported()) return BAKRON_ERR_UNSUPPORTED;
  return launch_status(grad ? launch_linear_tc(a, grad, s) : launch_linear_fwd(a, s));
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_linear_workspace_size(const bakron_packed* w, int64_t T, int dtype,
                                                      size_t* bytes) {
  LinearArgs a;
  if (!bytes || !linear_args(w, T, dtype, w, w, &a)) return BAKRON_ERR_INVALID_ARG;
  *bytes = workspace_bytes(a, false);
  return BAKRON_OK;
}

extern "C" bakron_status bakron_linear(const void* X, int64_t T, int dtype, const bakron_packed* w,
                                       void* Y, void* ws, size_t ws_bytes, void* stream) {
  LinearArgs a;
  if (!linear_args(X, T, dtype, w, Y, &a)) return BAKRON_ERR_INVALID_ARG;
  return run_linear(a, false, ws, ws_bytes, stream);
}

extern "C" bakron_status bakron_linear_grad_workspace_size(const bakron_packed* w, int64_t T,
                                                           int dtype, size_t* bytes) {
  LinearArgs a;
  if (!bytes || !linear_args(w, T, dtype, w, w, &a)) return BAKRON_ERR_INVALID_ARG;
  *bytes = workspace_bytes(a, true);
  return BAKRON_OK;
}

extern "C" bakron_status bakron_linear_grad(const void* dY, int64_t T, int dtype,
                                            const bakron_packed* w, void* dX, void* ws,
                                            size_t ws_bytes, void* stream) {
  LinearArgs a;
  if (!linear_args(dY, T, dtype, w, dX, &a)) return BAKRON_ERR_INVALID_ARG;
  return run_linear(a, true, ws, ws_bytes, stream);
}
