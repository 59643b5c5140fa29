// Entry points of the quantised linear layer: argument checks and the choice
// of kernel.
#include <algorithm>

#include "linear_tc.cuh"

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
                 LinearArgs* a, bool experts = false) {
  if (!dtype_ok(dtype) || T < 0 || T > (int64_t(1) << 28) || !packed_view(w, &a->w)) return false;
  if (!experts && a->w.count != 1) return false;
  if (T > 0 && (!x || !y || !aligned_to(x, dtype_size(dtype)) || !aligned_to(y, dtype_size(dtype))))
    return false;
  a->x = x;
  a->y = const_cast<void*>(y);
  a->T = T;
  a->dtype = dtype;
  a->epi = {};
  a->offsets = nullptr;
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
  if (a.T > kMidTokens) return kMany;
  // About microseconds, the second by the codes and the columns, the third by the chunks of a block, which cost
  // more when they hold more groups or zero points; fitted to what is faster (11 shapes from 1024 x 1024 to
  // 8192 x 8192, 128 x 16384 and 14336 x 4096, 17 to 64 tokens, groups of 128, 64 and 32: 9 of 462 calls more than 10 %
  // from the faster one).  Second and third: 32 tokens of 8192 x 8192 in groups of 128 24.5 and 20.5, 64 29.6 and 22.4,
  // 32 29.7 and 38.6; 48 tokens of 4096 x 4096 11.6 and 10.8, 13.6 and 10.5, 13.6 and 13.8; of 1000 x 4096
  // 7.1 and 8.3, 8.3 and 7.5, 8.3 and 9.2.
  const bool narrow = a.w.ng > 1 && a.w.g % 128 != 0;
  const double work = 1e-6 * (double)(a.w.mp * a.w.nc * 128) + 0.28 * (double)a.w.nc;
  const double mid = a.T <= 32   ? (narrow ? 2.8 + work * 0.275 : 3.5 + work * 0.227)
                     : a.T <= 48 ? 4.3 + work * (narrow ? 0.44 : 0.27)
                                 : (narrow ? 7.0 + work * 0.47 : 5.1 + work * 0.353);
  const double chunk = !narrow ? 0.35 : a.w.g % 64 == 0 ? 0.33 : 0.87;
  const double many = 6.7 + (double)linear_fwd_steps(a) * chunk * (a.w.zero && a.w.g % 64 == 0 ? 1.25 : 1.0);
  return mid < many ? kMid : kMany;
}

size_t workspace_bytes(const LinearArgs& a, bool grad, bool experts = false) {
  if (!grad && !experts && a.T <= kFewTokens && forward_kernel(a) == kFew) return 0;
  if (grad && a.dtype != BAKRON_F32 && a.w.m > grad_chain(a.dtype) && a.T > 0)
    return grad_planes_bytes(a) +
           (size_t)sm_count() * (size_t)std::min<int64_t>(kGradTokens, (a.T + 31) / 32 * 32) * 128 * sizeof(float);
  const int64_t K = grad ? a.w.m : a.w.n;
  return (size_t)(a.dtype == BAKRON_F32 ? 3 : 1) * (size_t)a.T * (size_t)((K + 127) / 128 * 128) * 2;
}

enum class Call { kLinear, kAct, kGrad };

bakron_status run_linear(LinearArgs& a, Call call, void* ws, size_t ws_bytes, void* stream) {
  if (a.T == 0) return BAKRON_OK;
  const bool grad = call == Call::kGrad, act = call == Call::kAct;
  const size_t need = workspace_bytes(a, grad);
  if (need > 0 && (!ws || !aligned_to(ws, 256) || ws_bytes < need)) return BAKRON_ERR_INVALID_ARG;
  a.ws = ws;
  cudaStream_t s = (cudaStream_t)stream;
  if (!grad) {
    const Kernel k = forward_kernel(a);
    if (k == kFew) return launch_status(act ? launch_linear_act_few(a, s) : launch_linear_few(a, s));
    if (k == kMid) return launch_status(act ? launch_linear_act_mid(a, s) : launch_linear_mid(a, s));
  }
  if (!prop_tc_supported()) return BAKRON_ERR_UNSUPPORTED;
  return launch_status(grad ? launch_linear_grad(a, s) : act ? launch_linear_act_fwd(a, s) : launch_linear_fwd(a, s));
}

// Experts' products: the rows of x that belong to them are known on the device alone, so
// the tcgen05 kernels take every number of rows.
bool experts_args(const void* x, int64_t R, int dtype, const bakron_packed* w, const int32_t* offsets,
                  const void* y, LinearArgs* a) {
  if (!linear_args(x, R, dtype, w, y, a, true) || a->w.count > kMaxGroupedExperts) return false;
  if (R > 0 && (!offsets || !aligned_to(offsets, 4))) return false;
  a->offsets = offsets;
  return true;
}

bakron_status run_experts(LinearArgs& a, bool grad, void* ws, size_t ws_bytes, void* stream) {
  if (a.T == 0) return BAKRON_OK;
  const size_t need = workspace_bytes(a, grad, true);
  if (!ws || !aligned_to(ws, 256) || ws_bytes < need) return BAKRON_ERR_INVALID_ARG;
  a.ws = ws;
  if (!prop_tc_supported()) return BAKRON_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  return launch_status(grad ? launch_experts_grad(a, s) : launch_experts_fwd(a, s));
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
  return run_linear(a, Call::kLinear, ws, ws_bytes, stream);
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
  return run_linear(a, Call::kGrad, ws, ws_bytes, stream);
}

extern "C" bakron_status bakron_linear_act(const void* X, int64_t T, int dtype, const bakron_packed* w,
                                           const float* bias, int act, const void* residual, void* Y,
                                           void* pre, void* ws, size_t ws_bytes, void* stream) {
  LinearArgs a;
  if (!linear_args(X, T, dtype, w, Y, &a) || !act_ok(act)) return BAKRON_ERR_INVALID_ARG;
  const size_t es = dtype_size(dtype);
  if (!aligned_to(bias, 4) || !aligned_to(residual, es) || !aligned_to(pre, es)) return BAKRON_ERR_INVALID_ARG;
  a.epi = {bias, residual, pre, act};
  return run_linear(a, Call::kAct, ws, ws_bytes, stream);
}

extern "C" bakron_status bakron_experts_workspace_size(const bakron_packed* w, int64_t R, int dtype, int grad,
                                                       size_t* bytes) {
  LinearArgs a;
  if (!bytes || (grad != 0 && grad != 1) || !experts_args(w, R, dtype, w, reinterpret_cast<const int32_t*>(w), w, &a))
    return BAKRON_ERR_INVALID_ARG;
  *bytes = workspace_bytes(a, grad != 0, true);
  return BAKRON_OK;
}

extern "C" bakron_status bakron_experts(const void* X, int64_t R, int dtype, const bakron_packed* w,
                                        const int32_t* offsets, void* Y, void* ws, size_t ws_bytes,
                                        void* stream) {
  LinearArgs a;
  if (!experts_args(X, R, dtype, w, offsets, Y, &a)) return BAKRON_ERR_INVALID_ARG;
  return run_experts(a, false, ws, ws_bytes, stream);
}

extern "C" bakron_status bakron_experts_grad(const void* dY, int64_t R, int dtype, const bakron_packed* w,
                                             const int32_t* offsets, void* dX, void* ws, size_t ws_bytes,
                                             void* stream) {
  LinearArgs a;
  if (!experts_args(dY, R, dtype, w, offsets, dX, &a)) return BAKRON_ERR_INVALID_ARG;
  return run_experts(a, true, ws, ws_bytes, stream);
}
