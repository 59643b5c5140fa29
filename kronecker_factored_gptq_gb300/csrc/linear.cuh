// Shared between the entry points of the quantised linear layer and its
// kernels.
#pragma once

#include "act.cuh"
#include "packed.cuh"

namespace bakron {

struct LinearArgs {
  const void* x;        // T x n (gradient: T x m)
  void* y;              // T x m (gradient: T x n)
  int64_t T;
  int dtype;
  PackedView w;
  void* ws;
  Epilogue epi;         // bakron_linear_act
  const int* offsets;   // experts: boundaries of their rows of x, w.count + 1
};

constexpr int kMaxGroupedExperts = 1024;      // of bakron_experts

// Tokens up to which bakron_linear may run linear_few_kernel and
// linear_mid_kernel.
constexpr int64_t kFewTokens = 16;
constexpr int64_t kMidTokens = 64;

// Rows of the gradient's sum (16-bit dY) that stay in one accumulator; more need
// room for it in the workspace, behind dY's planes: N x 128 floats per block.
__host__ __device__ constexpr int64_t grad_chain(int dtype) { return dtype == BAKRON_F16 ? 4096 : 32768; }
constexpr int64_t kGradTokens = 256;     // N at most
inline size_t grad_planes_bytes(const LinearArgs& a) {
  const size_t b = (size_t)(a.dtype == BAKRON_F32 ? 3 : 1) * (size_t)a.T * (size_t)((a.w.m + 127) / 128 * 128) * 2;
  return (b + 255) / 256 * 256;
}

cudaError_t launch_linear_few(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_linear_mid(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_linear_act_few(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_linear_act_mid(const LinearArgs& a, cudaStream_t s);

// x (T x K of dtype, any alignment) -> planes [terms][T][kp] of 16-bit terms (1,
// or 3 for fp32), zeros past K; out is 16-byte aligned, kp a multiple of 8.  `grad`: the
// terms of the gradient's dY (split3_grad).
cudaError_t launch_planes(const void* x, int dtype, int64_t T, int64_t K, int64_t kp, void* out,
                          cudaStream_t s, bool grad = false);

// tcgen05 products for many tokens, and the gradient for any number.
cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t s);
int64_t linear_fwd_steps(const LinearArgs& a);    // 128-column chunks that its busiest block takes (16-bit x)
int linear_fwd_eights();                          // clusters of eight of its blocks that the current device runs at once
cudaError_t launch_linear_grad(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_linear_act_fwd(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_experts_fwd(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_experts_grad(const LinearArgs& a, cudaStream_t s);

}  // namespace bakron
