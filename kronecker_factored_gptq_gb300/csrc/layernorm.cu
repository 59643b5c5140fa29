// Layer norm over rows and its gradients.
//
// Forward: mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + eps),
// y = (x - mu) r gamma + beta.  Backward, with h = (x - mu) r, a = dy gamma:
//   dx = r (a - mean(a) - h mean(a h)),  dgamma = sum_t dy h,  dbeta = sum_t dy.
// Both are bound by HBM: forward reads and writes each element once, backward
// reads two and writes one.  A row stays in registers between its reductions
// (the variance from the deviations, not from a difference of two large
// sums), so nothing is read twice: one warp per row while a warp's registers
// hold it, else one block per row.  A thread owns the same columns of
// every row that its block takes, so the sums over rows of dgamma and dbeta
// grow in registers and leave the block once, into a row of the workspace; a
// second launch adds the blocks' rows in a fixed order (no atomics, so the
// bits do not depend on the run).
#include <algorithm>

#include "packed.cuh"

namespace bakron {
namespace {

struct NormArgs {
  const void* x;
  const void* dy;
  int64_t T, d;
  const float* gamma;
  const float* beta;
  float eps;
  void* y;               // y, or dx
  float* mean;
  float* rstd;
  const float* mean_in;
  const float* rstd_in;
  float* part;           // [blocks][2][d], NULL without weight gradients
};

constexpr int kMaxWarps = 32;

// Sum of (a, b) over the threads that share a row: the warp, or the block.
// `slot` alternates between calls, so one barrier per call is enough: a
// slot is written again only after the barrier of the call in between.
template <bool kBlock>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2 (*red)[kMaxWarps], int& slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if constexpr (kBlock) {
    if ((threadIdx.x & 31) == 0) red[slot][threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const int nw = blockDim.x >> 5;
    a = b = 0.f;
    for (int w = 0; w < nw; ++w) {
      const float2 v = red[slot][w];
      a += v.x;
      b += v.y;
    }
    slot ^= 1;
  }
}

// V consecutive elements.
template <typename TX, int V>
struct alignas(sizeof(TX) * V) Vec {
  TX v[V];
};

template <typename TX, int V, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256) norm_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float2 red[2][kMaxWarps];
  int slot = 0;
  const int tid = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int tpr = kBlock ? blockDim.x : 32;
  const int rows_at_once = kBlock ? 1 : blockDim.x >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * rows_at_once + (kBlock ? 0 : threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * rows_at_once;
  const float inv_d = 1.f / (float)p.d;
  for (int64_t row = row0; row < p.T; row += step) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    TX* y = static_cast<TX*>(p.y) + row * p.d;
    float f[NV][V];
    float sum = 0.f, sq = 0.f, unused = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
        const Vec<TX, V> v = *reinterpret_cast<const Vec<TX, V>*>(x + c);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[i][e] = to_float(v.v[e]);
          sum += f[i][e];
        }
      }
    }
    row_sum2<kBlock>(sum, unused, red, slot);
    const float mu = sum * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[i][e] -= mu;
          sq = fmaf(f[i][e], f[i][e], sq);
        }
      }
    }
    row_sum2<kBlock>(sq, unused, red, slot);
    const float r = 1.f / sqrtf(sq * inv_d + p.eps);
    if (tid == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
        Vec<TX, V> o;
        Vec<float, V> g, b;
        if (p.gamma) g = *reinterpret_cast<const Vec<float, V>*>(p.gamma + c);
        if (p.beta) b = *reinterpret_cast<const Vec<float, V>*>(p.beta + c);
#pragma unroll
        for (int e = 0; e < V; ++e)
          o.v[e] = from_float<TX>(fmaf(f[i][e] * r, p.gamma ? g.v[e] : 1.f, p.beta ? b.v[e] : 0.f));
        *reinterpret_cast<Vec<TX, V>*>(y + c) = o;
      }
    }
  }
}

template <typename TX, int V, int NV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 1024 : 256)
    norm_grad_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float2 red[2][kMaxWarps];
  int slot = 0;
  const int tid = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int tpr = kBlock ? blockDim.x : 32;
  const int rows_at_once = kBlock ? 1 : blockDim.x >> 5;
  const int64_t lead = (int64_t)blockIdx.x * rows_at_once + (kBlock ? 0 : threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * rows_at_once;
  const float inv_d = 1.f / (float)p.d;
  float dg[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dg[i][e] = db[i][e] = 0.f;
  for (int64_t row = lead; row < p.T; row += step) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    const TX* dy = static_cast<const TX*>(p.dy) + row * p.d;
    TX* dx = static_cast<TX*>(p.y) + row * p.d;
    const float mu = p.mean_in[row], r = p.rstd_in[row];
    Vec<TX, V> vx[NV], vy[NV];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
        vx[i] = *reinterpret_cast<const Vec<TX, V>*>(x + c);
        vy[i] = *reinterpret_cast<const Vec<TX, V>*>(dy + c);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
        Vec<float, V> g;
        if (p.gamma) g = *reinterpret_cast<const Vec<float, V>*>(p.gamma + c);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float h = (to_float(vx[i].v[e]) - mu) * r, d = to_float(vy[i].v[e]);
          const float a = d * (p.gamma ? g.v[e] : 1.f);
          s1 += a;
          s2 = fmaf(a, h, s2);
          dg[i][e] = fmaf(d, h, dg[i][e]);
          db[i][e] += d;
        }
      }
    }
    row_sum2<kBlock>(s1, s2, red, slot);
    s1 *= inv_d;
    s2 *= inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
        Vec<TX, V> o;
        Vec<float, V> g;
        if (p.gamma) g = *reinterpret_cast<const Vec<float, V>*>(p.gamma + c);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float h = (to_float(vx[i].v[e]) - mu) * r;
          const float a = to_float(vy[i].v[e]) * (p.gamma ? g.v[e] : 1.f);
          o.v[e] = from_float<TX>(r * (a - s1 - h * s2));
        }
        *reinterpret_cast<Vec<TX, V>*>(dx + c) = o;
      }
    }
  }
  if (p.part) {
    // one row of partial sums per block, or per warp
    float* o = p.part + lead * 2 * p.d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          o[c + e] = dg[i][e];
          o[p.d + c + e] = db[i][e];
        }
      }
    }
  }
}

// Rows too long for a block's registers: the row is read again from memory
// (mostly from L2) for each reduction, and the partial weight gradients live
// in the block's row of the workspace, where only one thread ever touches a
// column.
template <typename TX>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float2 red[2][kMaxWarps];
  int slot = 0;
  const float inv_d = 1.f / (float)p.d;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    TX* y = static_cast<TX*>(p.y) + row * p.d;
    float sum = 0.f, sq = 0.f, unused = 0.f;
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) sum += to_float(x[c]);
    row_sum2<true>(sum, unused, red, slot);
    const float mu = sum * inv_d;
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float v = to_float(x[c]) - mu;
      sq = fmaf(v, v, sq);
    }
    row_sum2<true>(sq, unused, red, slot);
    const float r = 1.f / sqrtf(sq * inv_d + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = mu;
      if (p.rstd) p.rstd[row] = r;
    }
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x)
      y[c] = from_float<TX>(fmaf((to_float(x[c]) - mu) * r, p.gamma ? p.gamma[c] : 1.f,
                                 p.beta ? p.beta[c] : 0.f));
  }
}

template <typename TX>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float2 red[2][kMaxWarps];
  int slot = 0;
  const float inv_d = 1.f / (float)p.d;
  float* o = p.part ? p.part + (int64_t)blockIdx.x * 2 * p.d : nullptr;
  if (o)
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) o[c] = o[p.d + c] = 0.f;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    const TX* dy = static_cast<const TX*>(p.dy) + row * p.d;
    TX* dx = static_cast<TX*>(p.y) + row * p.d;
    const float mu = p.mean_in[row], r = p.rstd_in[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float h = (to_float(x[c]) - mu) * r, d = to_float(dy[c]);
      const float a = d * (p.gamma ? p.gamma[c] : 1.f);
      s1 += a;
      s2 = fmaf(a, h, s2);
      if (o) {
        o[c] = fmaf(d, h, o[c]);
        o[p.d + c] += d;
      }
    }
    row_sum2<true>(s1, s2, red, slot);
    s1 *= inv_d;
    s2 *= inv_d;
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float h = (to_float(x[c]) - mu) * r;
      const float a = to_float(dy[c]) * (p.gamma ? p.gamma[c] : 1.f);
      dx[c] = from_float<TX>(r * (a - s1 - h * s2));
    }
  }
}

// dgamma and dbeta: the sum over the partial rows.  A block takes 32 columns,
// its 16 warps every 16th row each, joined in shared memory in a fixed order.
__global__ void __launch_bounds__(512) norm_join_kernel(const float* __restrict__ part, int64_t rows,
                                                        int64_t d, float* __restrict__ dgamma,
                                                        float* __restrict__ dbeta) {
  __shared__ float red[16][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;      // over 2 d columns
  float v = 0.f;
  if (c < 2 * d) {
#pragma unroll 4
    for (int64_t r = warp; r < rows; r += 16) v += part[r * 2 * d + c];
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < 2 * d) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    if (c < d) dgamma[c] = s;
    else dbeta[c - d] = s;
  }
}

// How a shape runs: vector width, vectors per thread, threads per row.
struct NormPlan {
  int v, nv;        // nv 0: the long-row kernels
  bool block;       // one block per row, else one warp
  int threads;      // of a block
};

NormPlan norm_plan(int64_t d, int dtype, bool aligned) {
  NormPlan q;
  const int wide = dtype == BAKRON_F32 ? 4 : 8;
  q.v = (aligned && d % wide == 0) ? wide : 1;
  const int64_t vecs = d / q.v;
  const int most = q.v == 1 ? 16 : 4;
  if (vecs <= 32 * most) {
    q.block = false;
    q.threads = 256;
    q.nv = most;
    return q;
  }
  q.block = true;
  if (vecs > (int64_t)1024 * most) {
    q.nv = 0;
    q.threads = 1024;
    return q;
  }
  q.nv = q.v == 1 ? most : vecs <= 256 ? 1 : vecs <= 512 ? 2 : 4;
  q.threads = (int)(((vecs + q.nv - 1) / q.nv + 31) / 32 * 32);
  return q;
}

int64_t fwd_blocks(const NormPlan& q, int64_t T) {
  const int rows = q.block ? 1 : q.threads / 32;
  return std::min<int64_t>((T + rows - 1) / rows, (int64_t)sm_count() * 32);
}

// Blocks of the backward launch.  Upper bound in the workspace size: the
// alignment of the pointers is not known there.
constexpr int kGradBlocksPerSm = 2;
int64_t grad_blocks(const NormPlan& q, int64_t T) {
  const int rows = q.block ? 1 : q.threads / 32;
  return std::min<int64_t>((T + rows - 1) / rows, (int64_t)sm_count() * kGradBlocksPerSm);
}
int64_t grad_rows(const NormPlan& q, int64_t T) {
  return grad_blocks(q, T) * (q.block ? 1 : q.threads / 32);
}

template <typename TX, int W>
cudaError_t run_fwd(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  const unsigned g = (unsigned)fwd_blocks(q, a.T);
  count_launch();
  if (q.nv == 0) norm_long_kernel<TX><<<g, q.threads, 0, s>>>(a);
  else if (q.v == 1 && !q.block) norm_kernel<TX, 1, 16, false><<<g, q.threads, 0, s>>>(a);
  else if (q.v == 1) norm_kernel<TX, 1, 16, true><<<g, q.threads, 0, s>>>(a);
  else if (!q.block) norm_kernel<TX, W, 4, false><<<g, q.threads, 0, s>>>(a);
  else if (q.nv == 1) norm_kernel<TX, W, 1, true><<<g, q.threads, 0, s>>>(a);
  else if (q.nv == 2) norm_kernel<TX, W, 2, true><<<g, q.threads, 0, s>>>(a);
  else norm_kernel<TX, W, 4, true><<<g, q.threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename TX, int W>
cudaError_t run_grad(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  const unsigned g = (unsigned)grad_blocks(q, a.T);
  count_launch();
  if (q.nv == 0) norm_grad_long_kernel<TX><<<g, q.threads, 0, s>>>(a);
  else if (q.v == 1 && !q.block) norm_grad_kernel<TX, 1, 16, false><<<g, q.threads, 0, s>>>(a);
  else if (q.v == 1) norm_grad_kernel<TX, 1, 16, true><<<g, q.threads, 0, s>>>(a);
  else if (!q.block) norm_grad_kernel<TX, W, 4, false><<<g, q.threads, 0, s>>>(a);
  else if (q.nv == 1) norm_grad_kernel<TX, W, 1, true><<<g, q.threads, 0, s>>>(a);
  else if (q.nv == 2) norm_grad_kernel<TX, W, 2, true><<<g, q.threads, 0, s>>>(a);
  else norm_grad_kernel<TX, W, 4, true><<<g, q.threads, 0, s>>>(a);
  return cudaGetLastError();
}

bool norm_args_ok(int64_t T, int64_t d, int dtype) {
  return dtype_ok(dtype) && T >= 0 && T <= (int64_t(1) << 31) && d >= 1 && d <= (int64_t(1) << 20);
}

size_t grad_bytes(int64_t T, int64_t d) {
  int64_t rows = 0;
  for (int dt : {BAKRON_F32, BAKRON_BF16})
    for (bool al : {false, true}) rows = std::max(rows, grad_rows(norm_plan(d, dt, al), T));
  return (size_t)(rows * 2 * d) * sizeof(float);
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_layernorm(const void* X, int64_t T, int64_t d, int dtype,
                                          const float* gamma, const float* beta, float eps, void* Y,
                                          float* mean, float* rstd, void* stream) {
  if (!norm_args_ok(T, d, dtype) || !(eps >= 0.f)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0) return BAKRON_OK;
  const size_t es = dtype_size(dtype);
  if (!X || !Y || !aligned_to(X, es) || !aligned_to(Y, es)) return BAKRON_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = X;
  a.T = T;
  a.d = d;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.y = Y;
  a.mean = mean;
  a.rstd = rstd;
  const bool al = aligned_to(X, 16) && aligned_to(Y, 16) && aligned_to(gamma, 32) && aligned_to(beta, 32);
  const NormPlan q = norm_plan(d, dtype, al);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == BAKRON_F32    ? run_fwd<float, 4>(q, a, s)
                        : dtype == BAKRON_BF16 ? run_fwd<__nv_bfloat16, 8>(q, a, s)
                                               : run_fwd<__half, 8>(q, a, s);
  return launch_status(e);
}

extern "C" bakron_status bakron_layernorm_grad_workspace_size(int64_t T, int64_t d, size_t* bytes) {
  if (!bytes || !norm_args_ok(T, d, BAKRON_F32)) return BAKRON_ERR_INVALID_ARG;
  *bytes = grad_bytes(T, d);
  return BAKRON_OK;
}

extern "C" bakron_status bakron_layernorm_grad(const void* dY, const void* X, int64_t T, int64_t d,
                                               int dtype, const float* gamma, const float* mean,
                                               const float* rstd, void* dX, float* dgamma,
                                               float* dbeta, void* ws, size_t ws_bytes,
                                               void* stream) {
  if (!norm_args_ok(T, d, dtype) || (dgamma == nullptr) != (dbeta == nullptr))
    return BAKRON_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    if (dgamma && (cudaMemsetAsync(dgamma, 0, (size_t)d * 4, s) != cudaSuccess ||
                   cudaMemsetAsync(dbeta, 0, (size_t)d * 4, s) != cudaSuccess))
      return BAKRON_ERR_CUDA;
    return BAKRON_OK;
  }
  const size_t es = dtype_size(dtype);
  if (!X || !dY || !dX || !mean || !rstd || !aligned_to(X, es) || !aligned_to(dY, es) ||
      !aligned_to(dX, es))
    return BAKRON_ERR_INVALID_ARG;
  if (dgamma && (!ws || !aligned_to(ws, 256) || ws_bytes < grad_bytes(T, d)))
    return BAKRON_ERR_INVALID_ARG;
  NormArgs a = {};
  a.x = X;
  a.dy = dY;
  a.T = T;
  a.d = d;
  a.gamma = gamma;
  a.y = dX;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.part = dgamma ? static_cast<float*>(ws) : nullptr;
  const bool al = aligned_to(X, 16) && aligned_to(dY, 16) && aligned_to(dX, 16) && aligned_to(gamma, 32);
  const NormPlan q = norm_plan(d, dtype, al);
  const cudaError_t e = dtype == BAKRON_F32    ? run_grad<float, 4>(q, a, s)
                        : dtype == BAKRON_BF16 ? run_grad<__nv_bfloat16, 8>(q, a, s)
                                               : run_grad<__half, 8>(q, a, s);
  if (e != cudaSuccess) return launch_status(e);
  if (dgamma) {
    count_launch();
    norm_join_kernel<<<(unsigned)((2 * d + 31) / 32), 512, 0, s>>>(a.part, grad_rows(q, T), d, dgamma,
                                                                     dbeta);
    if (cudaGetLastError() != cudaSuccess) return BAKRON_ERR_CUDA;
  }
  return BAKRON_OK;
}
