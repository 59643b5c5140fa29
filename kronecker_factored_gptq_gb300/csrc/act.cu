// bakron_act and bakron_act_grad: y = a(z), dz = dy a'(z), db = sum_t dz_t; gated: y = a(g) u,
// dg = dy u a'(g), du = dy a(g).
//
// Elementwise, so bound by the bytes of z, dy and the results, each met once.  A block's
// threads are cx columns (of V elements, 16 bytes where the rows allow) by 256 / cx rows,
// and a thread keeps its columns for all its rows, so that the bias's gradient grows in
// registers; kRows rows are loaded before the first is used.  A block's column sums are
// joined in shared memory and go to its row of the workspace, which a second launch adds up in
// a fixed order (no atomics: the bits do not depend on the run); with one block of rows they
// are the result.  The activation is chosen once for a thread's rows at hand, not per value.
// Measured, gated silu of 2048 x 14336 bf16: 31 us (the bytes at 6.80 TB/s: 26), its gradient 48 (43); exact gelu, whose
// erfcf is longer than the bytes, 56 and 69 (not gated 52 and 66; relu 21 and 29); 37 x 1111
// fp32 gelu 2.6 and with the bias's gradient 3.0 us: launch and latency.  Rows that do not begin on 16 bytes go
// by pieces of 8, 4 or 2 bytes (2048 x 6144 bf16 silu 12 us; 6148, 6146 and 6145 columns 13, 16 and 24).
#include <algorithm>

#include "act.cuh"
#include "piece.cuh"

namespace bakron {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxColumns = int64_t(1) << 20;

struct ActArgs {
  const void* z;
  const void* dy;
  void* out;            // y, or dz
  int64_t T, m;
  int act, cx;          // cx: threads along the columns, a power of two
  float* sums;          // [row blocks][columns of z], or dbias
};

template <typename TX, int V, bool kGated, bool kGrad, bool kSums>
__global__ void __launch_bounds__(kThreads, kSums ? 3 : 4) act_kernel(const __grid_constant__ ActArgs a) {
  using W = Piece<TX, V * (int)sizeof(TX)>;
  // rows at hand: more of narrow pieces (2048 x 6146 bf16 24 us with four, 16), but of single elements whose
  // columns are summed (2048 x 6145: 38 us with eight, 33)
  constexpr int VB = V * (int)sizeof(TX);
  constexpr int kRows = VB == 16 ? (kGated ? 2 : 4) : VB == 8 || (V == 1 && kSums) ? 4 : 8;
  constexpr int NS = kSums ? (kGated ? 2 : 1) * V : 1;
  const int tx = threadIdx.x & (a.cx - 1), ty = threadIdx.x / a.cx, ry = kThreads / a.cx;
  const int64_t col = ((int64_t)blockIdx.x * a.cx + tx) * V;
  const int64_t zc = kGated ? 2 * a.m : a.m;
  const int64_t r1 = a.T * (blockIdx.y + 1) / gridDim.y;
  const TX* z = static_cast<const TX*>(a.z) + col;
  const TX* dy = static_cast<const TX*>(a.dy) + col;
  TX* out = static_cast<TX*>(a.out) + col;
  const int64_t oc = kGrad ? zc : a.m;
  float sum[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) sum[i] = 0.f;
  if (col < a.m) {
    for (int64_t r = a.T * blockIdx.y / gridDim.y + ty; r < r1; r += (int64_t)kRows * ry) {
      W g[kRows], u[kRows], d[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t row = r + (int64_t)i * ry;
        if (row < r1) {
          g[i] = *reinterpret_cast<const W*>(z + row * zc);
          if constexpr (kGated) u[i] = *reinterpret_cast<const W*>(z + row * zc + a.m);
          if constexpr (kGrad) d[i] = *reinterpret_cast<const W*>(dy + row * a.m);
        }
      }
      by_act(a.act, [&](auto A) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const int64_t row = r + (int64_t)i * ry;
          if (row < r1) {
            W o;
            float vo[V], vp[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float x = g[i].get(e);
              if constexpr (!kGrad) {
                float y = activate<TX, A>(x);
                if constexpr (kGated) y *= u[i].get(e);
                vo[e] = y;
              } else {
                float f, slope;
                activate_slope<TX, A>(x, f, slope);
                float q = d[i].get(e);
                if constexpr (kGated) {
                  const float t = q * f;
                  vp[e] = t;
                  if constexpr (kSums) sum[V + e] += t;
                  q *= u[i].get(e);
                }
                q *= slope;
                vo[e] = q;
                if constexpr (kSums) sum[e] += q;
              }
            }
            o.set(vo);
            *reinterpret_cast<W*>(out + row * oc) = o;
            if constexpr (kGated && kGrad) {
              o.set(vp);
              *reinterpret_cast<W*>(out + row * oc + a.m) = o;
            }
          }
        }
      });
    }
  }
  if constexpr (kSums) {
    __shared__ float red[NS][kThreads];
#pragma unroll
    for (int i = 0; i < NS; ++i) red[i][threadIdx.x] = sum[i];
    __syncthreads();
    // thread i: value i / cx of column i % cx
    for (int i = threadIdx.x; i < NS * a.cx; i += kThreads) {
      const int c = i & (a.cx - 1), n = i / a.cx;
      float v = 0.f;
      for (int y = 0; y < ry; ++y) v += red[n][y * a.cx + c];
      const int64_t at = ((int64_t)blockIdx.x * a.cx + c) * V + n % V;
      if (at < a.m) a.sums[blockIdx.y * zc + (n / V) * a.m + at] = v;
    }
  }
}

// dbias: the sum over the row blocks, 16 warps every 16th row each for 32 columns.
__global__ void __launch_bounds__(512) act_join_kernel(const float* __restrict__ sums, int rows, int64_t columns,
                                                       float* __restrict__ dbias) {
  __shared__ float red[16][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < columns) {
#pragma unroll 4
    for (int r = warp; r < rows; r += 16) v += __ldcg(sums + r * columns + c);
  }
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < columns) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += red[w][lane];
    dbias[c] = s;
  }
}

// Row blocks: as many as fill the SMs eight times, but four rows for each thread at least, and one
// block as long as a thread then has eight at most: a second launch, which joins the blocks' sums,
// costs more (37 x 1111 fp32).
struct Grid {
  int cx;
  int64_t strips, blocks;
};
Grid act_grid(int64_t T, int64_t m, int V) {
  Grid g;
  const int64_t vecs = (m + V - 1) / V;
  g.cx = 1;
  while (g.cx < 32 && g.cx < vecs) g.cx *= 2;
  g.strips = (vecs + g.cx - 1) / g.cx;
  const int64_t rows = (int64_t)4 * (kThreads / g.cx);
  if (T <= 2 * rows) {
    g.blocks = 1;
    return g;
  }
  g.blocks = std::max<int64_t>(1, std::min<int64_t>((T + rows - 1) / rows, (int64_t)sm_count() * 8 / g.strips));
  return g;
}

template <typename TX, int V, bool kGated>
cudaError_t launch_act(ActArgs& a, bool grad, float* dbias, cudaStream_t s) {
  const Grid g = act_grid(a.T, a.m, V);
  a.cx = g.cx;
  const dim3 grid((unsigned)g.strips, (unsigned)g.blocks);
  count_launch();
  if (!grad) {
    act_kernel<TX, V, kGated, false, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (!dbias) {
    act_kernel<TX, V, kGated, true, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  float* const part = a.sums;
  if (g.blocks == 1) a.sums = dbias;
  act_kernel<TX, V, kGated, true, true><<<grid, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || g.blocks == 1) return e;
  const int64_t columns = kGated ? 2 * a.m : a.m;
  count_launch();
  act_join_kernel<<<(unsigned)((columns + 31) / 32), 512, 0, s>>>(part, (int)g.blocks, columns, dbias);
  return cudaGetLastError();
}

template <typename TX, int V>
cudaError_t by_gate(ActArgs& a, bool gated, bool grad, float* dbias, cudaStream_t s) {
  return gated ? launch_act<TX, V, true>(a, grad, dbias, s) : launch_act<TX, V, false>(a, grad, dbias, s);
}

template <typename TX>
cudaError_t by_vector(ActArgs& a, bool gated, bool grad, float* dbias, cudaStream_t s) {
  // the widest pieces that rows and addresses allow
  const uintptr_t all = (uintptr_t)(a.m * (int64_t)sizeof(TX)) | reinterpret_cast<uintptr_t>(a.z) |
                        reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.dy);
  constexpr int E = (int)sizeof(TX);
  if (all % 16 == 0) return by_gate<TX, 16 / E>(a, gated, grad, dbias, s);
  if (all % 8 == 0) return by_gate<TX, 8 / E>(a, gated, grad, dbias, s);
  if constexpr (E == 2) {
    if (all % 4 == 0) return by_gate<TX, 2>(a, gated, grad, dbias, s);
  }
  return by_gate<TX, 1>(a, gated, grad, dbias, s);
}

cudaError_t run_act(ActArgs& a, int dtype, bool gated, bool grad, float* dbias, cudaStream_t s) {
  switch (dtype) {
    case BAKRON_F32: return by_vector<float>(a, gated, grad, dbias, s);
    case BAKRON_BF16: return by_vector<__nv_bfloat16>(a, gated, grad, dbias, s);
    default: return by_vector<__half>(a, gated, grad, dbias, s);
  }
}

bool act_args_ok(int64_t T, int64_t m, int dtype, int act, int gated) {
  return dtype_ok(dtype) && act_ok(act) && (gated == 0 || gated == 1) && T >= 0 && T <= (int64_t(1) << 28) && m >= 1 &&
         m <= kMaxColumns;
}

// Neither the type, the alignment nor the gate is known to the size call; fewer rows never take more.
size_t act_grad_bytes(int64_t T, int64_t columns) {
  int64_t blocks = 0;
  for (int64_t m : {columns, (columns + 1) / 2})
    for (int V : {1, 2, 4, 8}) blocks = std::max(blocks, act_grid(T, m, V).blocks);
  return blocks > 1 ? (size_t)(blocks * columns) * sizeof(float) : 0;
}

}  // namespace
}  // namespace bakron

using namespace bakron;

extern "C" bakron_status bakron_act(const void* Z, int64_t T, int64_t m, int dtype, int act, int gated, void* Y,
                                    void* stream) {
  if (!act_args_ok(T, m, dtype, act, gated)) return BAKRON_ERR_INVALID_ARG;
  if (T == 0) return BAKRON_OK;
  const size_t es = dtype_size(dtype);
  if (!Z || !Y || !aligned_to(Z, es) || !aligned_to(Y, es)) return BAKRON_ERR_INVALID_ARG;
  ActArgs a = {};
  a.z = Z;
  a.out = Y;
  a.T = T;
  a.m = m;
  a.act = act;
  return launch_status(run_act(a, dtype, gated != 0, false, nullptr, (cudaStream_t)stream));
}

extern "C" bakron_status bakron_act_grad_workspace_size(int64_t T, int64_t columns, size_t* bytes) {
  if (!bytes || T < 0 || T > (int64_t(1) << 28) || columns < 1 || columns > 2 * kMaxColumns)
    return BAKRON_ERR_INVALID_ARG;
  *bytes = act_grad_bytes(T, columns);
  return BAKRON_OK;
}

extern "C" bakron_status bakron_act_grad(const void* dY, const void* Z, int64_t T, int64_t m, int dtype, int act,
                                         int gated, void* dZ, float* dbias, void* ws, size_t ws_bytes,
                                         void* stream) {
  if (!act_args_ok(T, m, dtype, act, gated) || !aligned_to(dbias, 4)) return BAKRON_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t columns = gated ? 2 * m : m;
  if (T == 0) {
    if (dbias && cudaMemsetAsync(dbias, 0, (size_t)columns * 4, s) != cudaSuccess) return BAKRON_ERR_CUDA;
    return BAKRON_OK;
  }
  const size_t es = dtype_size(dtype);
  if (!Z || !dY || !dZ || !aligned_to(Z, es) || !aligned_to(dY, es) || !aligned_to(dZ, es)) return BAKRON_ERR_INVALID_ARG;
  if (dbias) {
    const size_t need = act_grad_bytes(T, columns);
    if (need > 0 && (!ws || !aligned_to(ws, 256) || ws_bytes < need)) return BAKRON_ERR_INVALID_ARG;
  }
  ActArgs a = {};
  a.z = Z;
  a.dy = dY;
  a.out = dZ;
  a.T = T;
  a.m = m;
  a.act = act;
  a.sums = static_cast<float*>(ws);
  return launch_status(run_act(a, dtype, gated != 0, true, dbias, s));
}
