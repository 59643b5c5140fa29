// Layer norm over rows and its gradients.
//
// Forward: mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + eps),
// y = (x - mu) r gamma + beta.  Backward, with h = (x - mu) r, a = dy gamma:
//   dx = r (a - mean(a) - h mean(a h)),  dgamma = sum_t dy h,  dbeta = sum_t dy.
// Both are bound by HBM: forward reads and writes each element once, backward
// reads two and writes one.  A row stays in registers between its reductions
// (the variance from the deviations, not from a difference of two large
// sums), so nothing is read twice: one warp per row while a warp's registers
// hold it, else one block per row.  A block's barriers leave the memory idle unless
// the rows after the one at hand are on their way, so the block-per-row kernels
// copy them asynchronously into shared memory, a few rows ahead; a thread
// copies what it reads itself, so the copies need no barrier.  A thread owns the
// same columns of every row that its block takes, so the sums over rows of
// dgamma and dbeta grow in registers and leave the block once, into a row of the
// workspace; a second launch adds the blocks' rows in a fixed order (no atomics,
// so the bits do not depend on the run).
#include <algorithm>
#include <type_traits>

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
  int depth;             // slots of rows in shared memory
};

constexpr int kMaxWarps = 32;

// Sums of N values over the threads that share a row: the warp, or the block.
// `slot` alternates between calls, so one barrier per call is enough: a
// slot is written again only after the barrier of the call in between.
template <bool kBlock, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[4][kMaxWarps], int& slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (kBlock) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) red[slot][k][threadIdx.x >> 5] = v[k];
    }
    __syncthreads();
    // every warp adds the warps' sums in the same way
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = lane < warps ? red[slot][k][lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o < warps) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
    slot ^= 1;
  }
}

// V consecutive elements.
template <typename TX, int V>
struct alignas(sizeof(TX) * V) Vec {
  TX v[V];
};

// The rows of a block (or warp) from memory, V elements at a time: loaded when
// asked for (kAhead false), or copied to shared memory `depth` - 1 rows ahead.
template <typename TX, int V, int NV, int ARRAYS, bool kAhead>
struct Rows {
  const TX* src[ARRAYS];
  int64_t d, step, T;
  int64_t next;             // next row to copy
  uint32_t slot, bytes;     // this thread's place in a slot; bytes of all slots
  uint32_t fill = 0, read = 0;
  int tid, tpr, depth;

  __device__ __forceinline__ uint32_t slot_bytes() const { return (uint32_t)(ARRAYS * NV * tpr) * 16u; }
  __device__ __forceinline__ void copy() {
    if (next < T) {
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (tid + i * tpr) * V;
          if (c < (int)d)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             slot + fill + (uint32_t)((k * NV + i) * tpr) * 16u),
                         "l"(src[k] + next * d + c)
                         : "memory");
        }
      next += step;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + slot_bytes() == bytes ? 0 : fill + slot_bytes();
  }
  __device__ __forceinline__ void start(int64_t first, void* smem) {
    if constexpr (kAhead) {
      next = first;
      bytes = slot_bytes() * (uint32_t)depth;
      slot = (uint32_t)__cvta_generic_to_shared(smem) + (uint32_t)tid * 16u +
             (tpr == 32 ? (threadIdx.x >> 5) * bytes : 0u);       // one row per warp, or per block
      for (int p = 0; p < depth - 1; ++p) copy();
    }
  }
  // Row `row`, the successor of the one asked for before.
  __device__ __forceinline__ void get(int64_t row, Vec<TX, V> (&v)[ARRAYS][NV]) {
    if constexpr (kAhead) {
      copy();
      // `depth` is 1 to 4
      if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
      else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
#pragma unroll
    for (int k = 0; k < ARRAYS; ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + i * tpr) * V;
        if (c < (int)d) {
          if constexpr (kAhead) {
            uint4 u;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                         : "r"(slot + read + (uint32_t)((k * NV + i) * tpr) * 16u)
                         : "memory");
            v[k][i] = *reinterpret_cast<const Vec<TX, V>*>(&u);
          } else {
            v[k][i] = *reinterpret_cast<const Vec<TX, V>*>(src[k] + row * d + c);
          }
        }
      }
    if constexpr (kAhead) read = read + slot_bytes() == bytes ? 0 : read + slot_bytes();
  }
};

// Two fp32 values at a time: one instruction for two additions, products or
// fused ones.  What bounds the block-per-row kernels after HBM is the number of
// instructions per element.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 f2(float v) { return F2{v, v}; }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("{\n .reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 r, a, b;\n"
      " mov.b64 {%0, %1}, r;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("{\n .reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 r, a, b;\n"
      " mov.b64 {%0, %1}, r;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("{\n .reg .b64 a, b, c, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 r, a, b, c;\n mov.b64 {%0, %1}, r;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// V elements to and from fp32, two at a time for the 16-bit types.
template <typename TX, int V>
__device__ __forceinline__ void widen(float (&f)[V], const Vec<TX, V>& v) {
  if constexpr (V > 1 && sizeof(TX) == 2) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      if constexpr (std::is_same<TX, __half>::value) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
      } else {
        f[2 * e] = __uint_as_float(u[e] << 16);
        f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = to_float(v.v[e]);
  }
}
template <typename TX, int V>
__device__ __forceinline__ void narrow(Vec<TX, V>& v, const float (&f)[V]) {
  if constexpr (V > 1 && sizeof(TX) == 2) {
    uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      if constexpr (std::is_same<TX, __half>::value) {
        const __half2 h = __floats2half2_rn(f[2 * e], f[2 * e + 1]);
        u[e] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        u[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v.v[e] = from_float<TX>(f[e]);
  }
}

// gamma and beta of V columns (1 and 0 where there are none).
template <int V>
__device__ __forceinline__ void params(Vec<float, V>& g, Vec<float, V>& b, const NormArgs& p, int c) {
  if (p.gamma && c < (int)p.d) {
    g = *reinterpret_cast<const Vec<float, V>*>(p.gamma + c);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) g.v[e] = 1.f;
  }
  if (p.beta && c < (int)p.d) {
    b = *reinterpret_cast<const Vec<float, V>*>(p.beta + c);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) b.v[e] = 0.f;
  }
}

template <typename TX, int V, int NV, bool kBlock, int MAXB>
__global__ void __launch_bounds__(MAXB, V == 1 && MAXB <= 512 ? 2 : 1) norm_kernel(const __grid_constant__ NormArgs p) {
  constexpr bool kAhead = V > 1;
  extern __shared__ __align__(16) uint8_t dsm[];
  __shared__ float red[2][4][kMaxWarps];
  int slot = 0;
  const int tid = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int tpr = kBlock ? blockDim.x : 32;
  const int rows_at_once = kBlock ? 1 : blockDim.x >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * rows_at_once + (kBlock ? 0 : threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * rows_at_once;
  const float inv_d = 1.f / (float)p.d;
  const int d = (int)p.d;
  Rows<TX, V, NV, 1, kAhead> rows;
  rows.src[0] = static_cast<const TX*>(p.x);
  rows.d = p.d;
  rows.step = step;
  rows.T = p.T;
  rows.tid = tid;
  rows.tpr = tpr;
  rows.depth = p.depth;
  rows.start(row0, dsm);
  // gamma and beta stay in registers when there is room
  constexpr bool kKeep = NV * V <= 16;
  Vec<float, V> gk[kKeep ? NV : 1], bk[kKeep ? NV : 1];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) params(gk[i], bk[i], p, (tid + i * tpr) * V);
  }
  // R rows at a time: their sums share the barriers and the shuffles' latency
  constexpr int R = kBlock && kAhead ? 2 : 1;
  for (int64_t row = row0; row < p.T; row += R * step) {
    float f[R][NV][V];
    float sum[R], sq[R];
    F2 p2[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      Vec<TX, V> v[1][NV];
      rows.get(row + q * step, v);
      sum[q] = sq[q] = 0.f;
      p2[q] = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if ((tid + i * tpr) * V < d) {
          widen(f[q][i], v[0][i]);
          if constexpr (V == 1) {
            sum[q] += f[q][i][0];
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) p2[q] = add2(p2[q], F2{f[q][i][e], f[q][i][e + 1]});
          }
        }
      }
      if constexpr (V > 1) sum[q] = p2[q].x + p2[q].y;
    }
    row_sums<kBlock, R>(sum, red, slot);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float mu = sum[q] * inv_d;
      sum[q] = mu;
      p2[q] = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if ((tid + i * tpr) * V < d) {
          if constexpr (V == 1) {
            f[q][i][0] -= mu;
            sq[q] = fmaf(f[q][i][0], f[q][i][0], sq[q]);
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const F2 t = add2(F2{f[q][i][e], f[q][i][e + 1]}, f2(-mu));
              p2[q] = fma2(t, t, p2[q]);
              f[q][i][e] = t.x;
              f[q][i][e + 1] = t.y;
            }
          }
        }
      }
      if constexpr (V > 1) sq[q] = p2[q].x + p2[q].y;
    }
    row_sums<kBlock, R>(sq, red, slot);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t at = row + q * step;
      if (at >= p.T) break;
      const float r = rsqrtf(sq[q] * inv_d + p.eps);
      if (tid == 0) {
        if (p.mean) p.mean[at] = sum[q];
        if (p.rstd) p.rstd[at] = r;
      }
      TX* y = static_cast<TX*>(p.y) + at * p.d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + i * tpr) * V;
        if (c < d) {
          if constexpr (!kKeep) params(gk[0], bk[0], p, c);
          const Vec<float, V>&g = gk[kKeep ? i : 0], &b = bk[kKeep ? i : 0];
          Vec<TX, V> o;
          if constexpr (V == 1) {
            f[q][i][0] = fmaf(f[q][i][0] * r, g.v[0], b.v[0]);
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const F2 t = fma2(mul2(F2{f[q][i][e], f[q][i][e + 1]}, f2(r)), F2{g.v[e], g.v[e + 1]},
                                F2{b.v[e], b.v[e + 1]});
              f[q][i][e] = t.x;
              f[q][i][e + 1] = t.y;
            }
          }
          narrow(o, f[q][i]);
          *reinterpret_cast<Vec<TX, V>*>(y + c) = o;
        }
      }
    }
  }
}

__device__ __forceinline__ float norm_h(float x, float mu, float r) { return (x - mu) * r; }

template <typename TX, int V, int NV, bool kBlock, int MAXB>
__global__ void __launch_bounds__(MAXB, MAXB <= 256 || V == 1 ? (MAXB <= 512 ? 2 : 1) : 1) norm_grad_kernel(const __grid_constant__ NormArgs p) {
  constexpr bool kAhead = V > 1;
  extern __shared__ __align__(16) uint8_t dsm[];
  __shared__ float red[2][4][kMaxWarps];
  int slot = 0;
  const int tid = kBlock ? threadIdx.x : threadIdx.x & 31;
  const int tpr = kBlock ? blockDim.x : 32;
  const int rows_at_once = kBlock ? 1 : blockDim.x >> 5;
  const int64_t lead = (int64_t)blockIdx.x * rows_at_once + (kBlock ? 0 : threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * rows_at_once;
  const float inv_d = 1.f / (float)p.d;
  const int d = (int)p.d;
  // gamma stays in registers when there is room
  constexpr bool kKeep = NV * V <= 16 && MAXB <= 512;
  Vec<float, V> gk[kKeep ? NV : 1], unused;
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) params(gk[i], unused, p, (tid + i * tpr) * V);
  }
  float dg[NV][V], db[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) dg[i][e] = db[i][e] = 0.f;
  Rows<TX, V, NV, 2, kAhead> rows;
  rows.src[0] = static_cast<const TX*>(p.x);
  rows.src[1] = static_cast<const TX*>(p.dy);
  rows.d = p.d;
  rows.step = step;
  rows.T = p.T;
  rows.tid = tid;
  rows.tpr = tpr;
  rows.depth = p.depth;
  rows.start(lead, dsm);
  // R rows at a time: their sums share the barrier and the shuffles' latency
  constexpr int R = kBlock && kAhead && MAXB <= 512 ? 2 : 1;
  float mu_next[R], r_next[R];
  auto stats = [&](int64_t row) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mu_next[q] = r_next[q] = 0.f;
      if (row + q * step < p.T) {
        mu_next[q] = ld_ahead(p.mean_in + row + q * step);
        r_next[q] = ld_ahead(p.rstd_in + row + q * step);
      }
    }
  };
  stats(lead);
  for (int64_t row = lead; row < p.T; row += R * step) {
    float mu[R], r[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      mu[q] = mu_next[q];
      r[q] = r_next[q];
    }
    stats(row + R * step);
    Vec<TX, V> v[R][2][NV];
    float sums[2 * R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      rows.get(row + q * step, v[q]);
      const bool there = row + q * step < p.T;
      float s1 = 0.f, s2 = 0.f;
      F2 t1 = f2(0.f), t2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + i * tpr) * V;
        if (c < d && there) {
          if constexpr (!kKeep) params(gk[0], unused, p, c);
          const Vec<float, V>& g = gk[kKeep ? i : 0];
          float fx[V], fw[V];
          widen(fx, v[q][0][i]);
          widen(fw, v[q][1][i]);
          if constexpr (V == 1) {
            const float h = norm_h(fx[0], mu[q], r[q]), w = fw[0], a = w * g.v[0];
            s1 += a;
            s2 = fmaf(a, h, s2);
            dg[i][0] = fmaf(w, h, dg[i][0]);
            db[i][0] += w;
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const F2 h = mul2(add2(F2{fx[e], fx[e + 1]}, f2(-mu[q])), f2(r[q])), w = F2{fw[e], fw[e + 1]};
              const F2 a = mul2(w, F2{g.v[e], g.v[e + 1]});
              t1 = add2(t1, a);
              t2 = fma2(a, h, t2);
              const F2 x = fma2(w, h, F2{dg[i][e], dg[i][e + 1]}), z = add2(F2{db[i][e], db[i][e + 1]}, w);
              dg[i][e] = x.x;
              dg[i][e + 1] = x.y;
              db[i][e] = z.x;
              db[i][e + 1] = z.y;
            }
          }
        }
      }
      sums[2 * q] = V > 1 ? t1.x + t1.y : s1;
      sums[2 * q + 1] = V > 1 ? t2.x + t2.y : s2;
    }
    row_sums<kBlock, 2 * R>(sums, red, slot);
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int64_t at = row + q * step;
      if (at >= p.T) break;
      TX* dx = static_cast<TX*>(p.y) + at * p.d;
      // dX = r a - (r m1) - h (r m2): three constants of the row
      const float m1 = r[q] * (sums[2 * q] * inv_d), m2 = r[q] * (sums[2 * q + 1] * inv_d);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (tid + i * tpr) * V;
        if (c < d) {
          if constexpr (!kKeep) params(gk[0], unused, p, c);
          const Vec<float, V>& g = gk[kKeep ? i : 0];
          Vec<TX, V> o;
          float fx[V], fw[V], fo[V];
          widen(fx, v[q][0][i]);
          widen(fw, v[q][1][i]);
          if constexpr (V == 1) {
            fo[0] = fmaf(-norm_h(fx[0], mu[q], r[q]), m2, fmaf(r[q], fw[0] * g.v[0], -m1));
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const F2 h = mul2(add2(F2{fx[e], fx[e + 1]}, f2(-mu[q])), f2(r[q]));
              const F2 a = mul2(F2{fw[e], fw[e + 1]}, F2{g.v[e], g.v[e + 1]});
              const F2 x = fma2(h, f2(-m2), fma2(a, f2(r[q]), f2(-m1)));
              fo[e] = x.x;
              fo[e + 1] = x.y;
            }
          }
          narrow(o, fo);
          *reinterpret_cast<Vec<TX, V>*>(dx + c) = o;
        }
      }
    }
  }
  if (!p.part) return;
  float* o = p.part + (int64_t)blockIdx.x * 2 * p.d;
  if constexpr (kBlock) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(tid + i * tpr) * V;
      if (c < p.d) {
        Vec<float, V> a, b;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          a.v[e] = dg[i][e];
          b.v[e] = db[i][e];
        }
        *reinterpret_cast<Vec<float, V>*>(o + c) = a;
        if constexpr (V == 1) o[p.d + c] = b.v[0];
        else *reinterpret_cast<Vec<float, V>*>(o + p.d + c) = b;
      }
    }
  } else {
    // the warps of the block add theirs one after the other, where the rows were
    float* sum = reinterpret_cast<float*>(dsm);     // [2][d]
    __syncthreads();
    for (int w = 0; w < rows_at_once; ++w) {
      if ((int)(threadIdx.x >> 5) == w) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const int64_t c = (int64_t)(tid + i * tpr) * V + e;
            if (c < p.d) {
              sum[c] = (w ? sum[c] : 0.f) + dg[i][e];
              sum[p.d + c] = (w ? sum[p.d + c] : 0.f) + db[i][e];
            }
          }
      }
      __syncthreads();
    }
    for (int64_t c = threadIdx.x; c < 2 * p.d; c += blockDim.x) o[c] = sum[c];
  }
}

// Rows too long for a block's registers: the row is read again from memory
// (mostly from L2) for each reduction, and the partial weight gradients live
// in the block's row of the workspace, where only one thread ever touches a
// column.
template <typename TX>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float red[2][4][kMaxWarps];
  int slot = 0;
  const float inv_d = 1.f / (float)p.d;
  for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x) {
    const TX* x = static_cast<const TX*>(p.x) + row * p.d;
    TX* y = static_cast<TX*>(p.y) + row * p.d;
    float sum[1] = {0.f}, sq[1] = {0.f};
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) sum[0] += to_float(x[c]);
    row_sums<true, 1>(sum, red, slot);
    const float mu = sum[0] * inv_d;
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float v = to_float(x[c]) - mu;
      sq[0] = fmaf(v, v, sq[0]);
    }
    row_sums<true, 1>(sq, red, slot);
    const float r = 1.f / sqrtf(sq[0] * inv_d + p.eps);
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
  __shared__ float red[2][4][kMaxWarps];
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
    float sums[2] = {0.f, 0.f};
    for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
      const float h = (to_float(x[c]) - mu) * r, d = to_float(dy[c]);
      const float a = d * (p.gamma ? p.gamma[c] : 1.f);
      sums[0] += a;
      sums[1] = fmaf(a, h, sums[1]);
      if (o) {
        o[c] = fmaf(d, h, o[c]);
        o[p.d + c] += d;
      }
    }
    row_sums<true, 2>(sums, red, slot);
    const float s1 = sums[0] * inv_d, s2 = sums[1] * inv_d;
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
#pragma unroll 8
    for (int64_t r = warp; r < rows; r += 16) v += __ldcg(part + r * 2 * d + c);
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

// How a shape runs: vector width, vectors per thread, threads per row, and for
// the block-per-row kernels the rows in flight.
struct NormPlan {
  int v, nv;        // nv 0: the long-row kernels
  bool block;       // one block per row, else one warp
  int threads;      // of a block
  int depth, per_sm;
  size_t smem;
};

// Shared memory per SM that the rows in flight may take (of 228 KB).
constexpr size_t kRowBytes = 200 * 1024;

NormPlan norm_plan(int64_t d, int dtype, bool aligned, int arrays) {
  NormPlan q = {};
  const int wide = dtype == BAKRON_F32 ? 4 : 8;
  q.v = (aligned && d % wide == 0) ? wide : 1;
  const int64_t vecs = d / q.v;
  // columns per thread: 32 forward, 16 backward (two sums per column live in
  // registers there), 32 once a block of 896 threads is too small for that; of
  // rows that are read by elements 8, or 16 for the longest
  const int most = q.v == 1 ? (vecs > 8 * 1024 ? 16 : 8)
                            : arrays == 1 || vecs > 16 / q.v * 896 ? 32 / q.v : 16 / q.v;
  if (vecs <= 32 * (q.v == 1 ? 8 : 32 / q.v)) {        // 256 odd columns, 1024 others: a warp per row
    q.threads = 256;
    q.nv = q.v == 1 ? 8 : 32 / q.v;
    q.per_sm = arrays == 1 ? 4 : 2;
    if (q.v > 1) {
      q.depth = 3;
      q.smem = (size_t)8 * q.depth * arrays * q.nv * 32 * 16;
    }
    if (arrays == 2) q.smem = std::max(q.smem, (size_t)(2 * d) * 4);    // the warps' sums
    return q;
  }
  q.block = true;
  if (vecs > (int64_t)1024 * most) {
    q.threads = 1024;
    q.per_sm = 2;
    return q;
  }
  q.nv = most;
  // a row of 32 threads would be taken for a warp's
  q.threads = std::max(64, (int)(((vecs + q.nv - 1) / q.nv + 31) / 32 * 32));
  if (q.v == 1) {
    q.per_sm = std::max(1, 1024 / q.threads);
    return q;
  }
  // blocks per SM: what the registers allow (128 a thread), fewer for long rows; as many rows
  // ahead as fit beside that
  const size_t row = (size_t)arrays * q.nv * q.threads * 16;
  q.per_sm = std::max(1, std::min(arrays == 1 ? 8 : 4, 512 / q.threads));
  while (q.per_sm > 1 && row * 2 * q.per_sm > kRowBytes) --q.per_sm;
  q.depth = (int)std::max<size_t>(1, std::min<size_t>(4, kRowBytes / (row * q.per_sm)));
  q.smem = row * q.depth;
  return q;
}

int64_t norm_blocks(const NormPlan& q, int64_t T) {
  const int rows = q.block ? 1 : q.threads / 32;
  return std::min<int64_t>((T + rows - 1) / rows, (int64_t)sm_count() * q.per_sm);
}

template <typename K>
cudaError_t launch_norm(K k, const NormPlan& q, const NormArgs& a, std::atomic<unsigned long long>& done,
                        cudaStream_t s) {
  if (q.smem > 46 * 1024) {      // beyond the default of 48 KB with the static part
    const cudaError_t e = ensure_smem_limit((const void*)k, 226 * 1024, done);
    if (e != cudaSuccess) return e;
  }
  count_launch();
  k<<<(unsigned)norm_blocks(q, a.T), q.threads, q.smem, s>>>(a);
  return cudaGetLastError();
}

template <typename TX, int W>
cudaError_t run_fwd(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  constexpr int N = 32 / W;
  static std::atomic<unsigned long long> d[8];
  if (q.nv == 0) return launch_norm(norm_long_kernel<TX>, q, a, d[0], s);
  if (q.v == 1 && !q.block) return launch_norm(norm_kernel<TX, 1, 8, false, 256>, q, a, d[1], s);
  if (q.v == 1 && q.threads <= 512) return launch_norm(norm_kernel<TX, 1, 8, true, 512>, q, a, d[2], s);
  if (q.v == 1 && q.nv == 8) return launch_norm(norm_kernel<TX, 1, 8, true, 1024>, q, a, d[7], s);
  if (q.v == 1) return launch_norm(norm_kernel<TX, 1, 16, true, 1024>, q, a, d[3], s);
  if (!q.block) return launch_norm(norm_kernel<TX, W, N, false, 256>, q, a, d[4], s);
  if (q.threads <= 512) return launch_norm(norm_kernel<TX, W, N, true, 512>, q, a, d[5], s);
  return launch_norm(norm_kernel<TX, W, N, true, 1024>, q, a, d[6], s);
}
template <typename TX, int W>
cudaError_t run_grad(const NormPlan& q, const NormArgs& a, cudaStream_t s) {
  constexpr int N = 16 / W;
  static std::atomic<unsigned long long> d[10];
  if (q.nv == 0) return launch_norm(norm_grad_long_kernel<TX>, q, a, d[0], s);
  if (q.v == 1 && !q.block) return launch_norm(norm_grad_kernel<TX, 1, 8, false, 256>, q, a, d[1], s);
  if (q.v == 1 && q.threads <= 512) return launch_norm(norm_grad_kernel<TX, 1, 8, true, 512>, q, a, d[2], s);
  if (q.v == 1 && q.nv == 8) return launch_norm(norm_grad_kernel<TX, 1, 8, true, 1024>, q, a, d[9], s);
  if (q.v == 1) return launch_norm(norm_grad_kernel<TX, 1, 16, true, 1024>, q, a, d[3], s);
  if (!q.block) return launch_norm(norm_grad_kernel<TX, W, 2 * N, false, 256>, q, a, d[4], s);
  if (q.nv == 2 * N) return launch_norm(norm_grad_kernel<TX, W, 2 * N, true, 1024>, q, a, d[5], s);
  if (q.threads <= 256) return launch_norm(norm_grad_kernel<TX, W, N, true, 256>, q, a, d[6], s);
  if (q.threads <= 512) return launch_norm(norm_grad_kernel<TX, W, N, true, 512>, q, a, d[7], s);
  return launch_norm(norm_grad_kernel<TX, W, N, true, 896>, q, a, d[8], s);
}

bool norm_args_ok(int64_t T, int64_t d, int dtype) {
  return dtype_ok(dtype) && T >= 0 && T <= (int64_t(1) << 31) && d >= 1 && d <= (int64_t(1) << 20);
}

// The alignment of the pointers and the type are not known to the size call.
size_t grad_bytes(int64_t T, int64_t d) {
  int64_t rows = 0;
  for (int dt : {BAKRON_F32, BAKRON_BF16})
    for (bool al : {false, true}) rows = std::max(rows, norm_blocks(norm_plan(d, dt, al, 2), T));
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
  const NormPlan q = norm_plan(d, dtype, al, 1);
  a.depth = q.depth;
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
  const NormPlan q = norm_plan(d, dtype, al, 2);
  a.depth = q.depth;
  const cudaError_t e = dtype == BAKRON_F32    ? run_grad<float, 4>(q, a, s)
                        : dtype == BAKRON_BF16 ? run_grad<__nv_bfloat16, 8>(q, a, s)
                                               : run_grad<__half, 8>(q, a, s);
  if (e != cudaSuccess) return launch_status(e);
  if (dgamma) {
    count_launch();
    norm_join_kernel<<<(unsigned)((2 * d + 31) / 32), 512, 0, s>>>(a.part, norm_blocks(q, T), d, dgamma,
                                                                     dbeta);
    if (cudaGetLastError() != cudaSuccess) return BAKRON_ERR_CUDA;
  }
  return BAKRON_OK;
}
