// Entry points of the quantised linear layer: argument checks and the choice
// of kernel.
#include <algorithm>

#include "linear.cuh"

namespace bakron {
namespace {

// Arguments both directions share; T = 0 is a valid call that does nothing.
bool linear_args(const void* x, int64_t T, int dtype, const bakron_packed* w, const void* y,
                 LinearArgs* a) {
  if (!dtype_ok(dtype) || T < 0 || T > (int64_t(1) << 31) || !packed_view(w, &a->w)) return false;
  if (a->w.count != 1) return false;
  if (T > 0 && (!x || !y || !aligned_to(x, dtype_size(dtype)) || !aligned_to(y, dtype_size(dtype))))
    return false;
  a->T = T;
  a->dtype = dtype;
  return true;
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_linear_workspace_size(const bakron_packed* w, int64_t T, int dtype,
                                                      size_t* bytes) {
  LinearArgs a;
  if (!bytes || !linear_args(w, T, dtype, w, w, &a)) return BAKRON_ERR_INVALID_ARG;
  *bytes = 0;
  return BAKRON_OK;
}

extern "C" bakron_status bakron_linear(const void* X, int64_t T, int dtype, const bakron_packed* w,
                                       void* Y, void* ws, size_t ws_bytes, void* stream) {
  LinearArgs a;
  if (!linear_args(X, T, dtype, w, Y, &a)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0) return BAKRON_OK;
  a.x = X;
  a.y = Y;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  return launch_linear_few(a, (cudaStream_t)stream) == cudaSuccess ? BAKRON_OK : BAKRON_ERR_CUDA;
}
