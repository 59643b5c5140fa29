// Entry points of the quantised linear layer: argument checks and the choice
// of kernel.
#include <algorithm>

#include "linear.cuh"

namespace bakron {
namespace {

// x (T x K, any alignment) -> planes [TERMS][T][kp] of 16-bit terms, zeros
// past K: the activations as the tensor map wants them.
template <typename TX, int TERMS, bool kGrad>
__global__ void __launch_bounds__(256) planes_kernel(const TX* __restrict__ x, int64_t T, int64_t K,
                                                     int64_t kp, uint16_t* __restrict__ out) {
  const int64_t per = kp / 8, total = T * per;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = i / per, k = (i - t * per) * 8;
    uint32_t h[TERMS][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t v[3] = {0, 0, 0};
      if (k + e < K) {
        const TX* p = x + t * K + k + e;
        if constexpr (TERMS == 1) {
          v[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
          float f[3];
          if constexpr (kGrad) split3_grad(to_float(*p), f[0], f[1], f[2]);
          else split3(to_float(*p), f[0], f[1], f[2]);
#pragma unroll
          for (int q = 0; q < 3; ++q) v[q] = bf16_bits(f[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < TERMS; ++q) h[q][e >> 1] = (e & 1) ? (h[q][e >> 1] | v[q] << 16) : v[q];
    }
#pragma unroll
    for (int q = 0; q < TERMS; ++q)
      *reinterpret_cast<uint4*>(out + (q * T + t) * kp + k) = make_uint4(h[q][0], h[q][1], h[q][2], h[q][3]);
  }
}

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

// Which forward kernel: a few tokens read in place (or staged at once, fp32)
// by blocks of 16 or 32 rows; more of them shared by larger blocks; the tcgen05
// kernel beyond.  fp32 tokens are three times the operand: at 8192 x 8192 and 8
// tokens the few-token kernel, staging them in parts, took 51 us, the second 23.
enum Kernel { kFew, kMid, kMany };
Kernel forward_kernel(const LinearArgs& a) {
  if (a.dtype == BAKRON_F32) {
    if (a.T > kFewTokens) return kMany;
    return a.T * a.w.nc * 128 * 6 <= 160 * 1024 ? kFew : kMid;
  }
  if (a.T <= kFewTokens) return kFew;
  if (a.T <= kMidTokens / 2) return kMid;
  if (a.T > kMidTokens) return kMany;
  // Between 33 and 64 tokens: microseconds by what was measured of the two, the
  // second by the codes, the third by a block's chunks, which cost more when
  // they hold more groups (bf16, second and third, groups of 128, 64 and 32;
  // 48 tokens of 8192 x 8192: 29.4 and 25.1, 41.5 and 39.2, 42.0 and 71.2; of 14336 x 4096,
  // whose 112 tiles leave SMs idle: 25.7 and 23.7, 31.6 and 38.2, 32.3 and 70.9; 64 tokens
  // of 8192 x 8192: 36.4 and 25.7, 55.3 and 39.8, 55.8 and 72.1).  Fitted to large
  // layers: of small ones it overrates the second (48 tokens of 4096 x 4096, groups of 64:
  // 13.7, and it takes the third's 14.9; of 2048 x 8192, groups of 128: 13.2 and 21.9).
  const bool narrow = a.w.ng > 1 && a.w.g % 128 != 0;
  const double mid = 1e-6 * (double)(a.w.mp * a.w.nc * 128) * (narrow ? 0.55 : 0.38) * (a.T <= 48 ? 1.0 : 1.3);
  const double many = (double)linear_fwd_steps(a) * (!narrow ? 0.57 : a.w.g % 64 == 0 ? 1.05 : 2.05);
  return mid < many ? kMid : kMany;
}

size_t workspace_bytes(const LinearArgs& a, bool grad) {
  if (!grad && a.T <= kFewTokens && forward_kernel(a) == kFew) return 0;
  if (grad && a.dtype != BAKRON_F32 && a.w.m > grad_chain(a.dtype) && a.T > 0)
    return grad_planes_bytes(a) +
           (size_t)sm_count() * (size_t)std::min<int64_t>(kGradTokens, (a.T + 31) / 32 * 32) * 128 * sizeof(float);
  const int64_t K = grad ? a.w.m : a.w.n;
  return (size_t)(a.dtype == BAKRON_F32 ? 3 : 1) * (size_t)a.T * (size_t)((K + 127) / 128 * 128) * 2;
}

bakron_status run_linear(LinearArgs& a, bool grad, void* ws, size_t ws_bytes, void* stream) {
  if (a.T == 0) return BAKRON_OK;
  const size_t need = workspace_bytes(a, grad);
  if (need > 0 && (!ws || !aligned_to(ws, 256) || ws_bytes < need)) return BAKRON_ERR_INVALID_ARG;
  a.ws = ws;
  cudaStream_t s = (cudaStream_t)stream;
  if (!grad) {
    const Kernel k = forward_kernel(a);
    if (k == kFew) return launch_status(launch_linear_few(a, s));
    if (k == kMid) return launch_status(launch_linear_mid(a, s));
  }
  if (!prop_tc_supported()) return BAKRON_ERR_UNSUPPORTED;
  return launch_status(grad ? launch_linear_grad(a, s) : launch_linear_fwd(a, s));
}

}  // namespace

cudaError_t launch_planes(const void* x, int dtype, int64_t T, int64_t K, int64_t kp, void* out,
                          cudaStream_t s, bool grad) {
  const int64_t total = T * kp / 8;
  const unsigned g = (unsigned)std::max<int64_t>(1, std::min<int64_t>((total + 255) / 256, (int64_t)sm_count() * 16));
  uint16_t* o = static_cast<uint16_t*>(out);
  count_launch();
  const float* f = static_cast<const float*>(x);
  if (dtype == BAKRON_F32 && grad) planes_kernel<float, 3, true><<<g, 256, 0, s>>>(f, T, K, kp, o);
  else if (dtype == BAKRON_F32) planes_kernel<float, 3, false><<<g, 256, 0, s>>>(f, T, K, kp, o);
  else planes_kernel<uint16_t, 1, false><<<g, 256, 0, s>>>(static_cast<const uint16_t*>(x), T, K, kp, o);
  return cudaGetLastError();
}

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
