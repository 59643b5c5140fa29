// bakron_linear for few tokens: Y = X V^T with X of up to a few dozen rows.
//
// y_ti = sum_k s_ik sum_{j in group k} x_tj (u_ij - z_ik).  Each code is read
// once and used for at most 16 tokens, so the codes' bytes bound the kernel
// (m n / 2; at 8192 x 8192 33.6 MB, 5.0 us at 6.68 TB/s); the products run on
// warp-level matrix instructions (qmma.cuh), which cost a fraction of that.
//
// A block takes 16 RB rows; its 8 warps take the 128-column chunks of the
// rows in turn, so that one block's loads in flight cover a long run of each
// row, and add their partial sums in shared memory in a fixed order.  Few
// rows leave SMs without a block: then the columns are also split over the
// blocks of a cluster, which are joined through distributed shared memory by
// the first of them, again in a fixed order.
#include <cooperative_groups.h>

#include <algorithm>

#include "linear.cuh"
#include "qmma.cuh"

namespace bakron {

namespace cg = cooperative_groups;

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr uint32_t kMaxXBytes = 96 * 1024;   // activations staged at a time

struct FewArgs {
  PackedView w;
  const void* x;
  void* y;
  int64_t T;
  int slab;      // chunks of activations staged at a time
  int vec_ok;    // rows of x are 16-byte aligned
};

template <typename TX, typename H, int TERMS, int NT, int RB, int NS>
__global__ void __launch_bounds__(kThreads) linear_few_kernel(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(16) uint8_t xs[];
  __shared__ float red[kWarps][NT * 8][16 * RB];
  __shared__ float part[NT * 8 * 16 * RB];
  cg::cluster_group cluster = cg::this_cluster();
  const int S = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)(blockIdx.x / S) * (16 * RB);
  const int64_t t0 = (int64_t)blockIdx.y * (8 * NT);
  const int cols = (int)min((int64_t)(8 * NT), a.T - t0);
  const TX* x = static_cast<const TX*>(a.x) + t0 * a.w.n;
  const int64_t c_lo = a.w.nc * rank / S, c_hi = a.w.nc * (rank + 1) / S;

  qm::TileRef tile[RB];
#pragma unroll
  for (int b = 0; b < RB; ++b) tile[b] = qm::tile_ref(a.w, 0, row0 + 16 * b, lane);
  int col[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) col[j] = min(8 * j + (lane >> 2), cols - 1);
  float tot[RB][NT][4];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[b][j][i] = 0.f;

  const uint32_t pitch = qm::x_pitch(a.slab);
  const uint32_t plane = pitch * (uint32_t)cols;
  qm::Chunk16<NS> f[RB];
  for (int64_t s0 = c_lo; s0 < c_hi; s0 += a.slab) {
    const int64_t s1 = min(s0 + a.slab, c_hi);
    int64_t c = s0 + warp;
    // the first codes are on their way while the activations are staged
    if (c < s1) {
#pragma unroll
      for (int b = 0; b < RB; ++b) qm::load_chunk<NS>(f[b], a.w, tile[b], c);
    }
    if (s0 != c_lo) __syncthreads();
    qm::stage_x<TX, TERMS>(xs, plane, pitch, x, a.w.n, cols, [](int r) { return (int64_t)r; },
                           s0 * 128, (int)(s1 - s0), a.w.n, a.vec_ok != 0);
    __syncthreads();
    for (; c < s1; c += kWarps) {
      qm::Chunk16<NS> g[RB];
      const bool more = c + kWarps < s1;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        g[b] = f[b];
        if (more) qm::load_chunk<NS>(f[b], a.w, tile[b], c + kWarps);
      }
      const uint8_t* xc = xs + (c - s0) * 256 + (lane & 3) * 16;
      qm::chunk_product<H, TERMS, RB, NT, NS>(
          tot, g, a.w.zero != nullptr, a.w.zu, NT, [&](int j, int q, int s) {
            return *reinterpret_cast<const uint4*>(xc + q * plane + (uint32_t)col[j] * pitch + s * 64);
          });
    }
  }

  // partial sums of the warps: [column][row], rows fastest
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = 16 * b + (lane >> 2), c = 8 * j + 2 * (lane & 3);
      red[warp][c][r] = tot[b][j][0];
      red[warp][c + 1][r] = tot[b][j][1];
      red[warp][c][r + 8] = tot[b][j][2];
      red[warp][c + 1][r + 8] = tot[b][j][3];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < NT * 8 * 16 * RB; i += kThreads) {
    const int c = i / (16 * RB), r = i - c * (16 * RB);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][c][r];
    if (S > 1) {
      part[i] = v;
    } else if (c < cols && row0 + r < a.w.m) {
      static_cast<TX*>(a.y)[(t0 + c) * a.w.m + row0 + r] = from_float<TX>(v);
    }
  }
  if (S > 1) {
    __syncwarp();
    cluster.sync();
    if (rank == 0) {
      for (int i = threadIdx.x; i < NT * 8 * 16 * RB; i += kThreads) {
        const int c = i / (16 * RB), r = i - c * (16 * RB);
        if (c >= cols || row0 + r >= a.w.m) continue;
        float v = 0.f;
        for (int k = 0; k < S; ++k) v += cluster.map_shared_rank(part, k)[i];
        static_cast<TX*>(a.y)[(t0 + c) * a.w.m + row0 + r] = from_float<TX>(v);
      }
    }
    __syncwarp();
    cluster.sync();   // no block leaves while its sums are read
  }
}

template <typename TX, typename H, int TERMS, int NT, int RB, int NS>
cudaError_t run(const LinearArgs& a, cudaStream_t s) {
  auto k = linear_few_kernel<TX, H, TERMS, NT, RB, NS>;
  FewArgs f;
  f.w = a.w;
  f.x = a.x;
  f.y = a.y;
  f.T = a.T;
  f.vec_ok = aligned_to(a.x, 16) && (a.w.n * sizeof(TX)) % 16 == 0;
  const int64_t tiles = (a.w.mp + 16 * RB - 1) / (16 * RB);
  const int64_t tt = (a.T + 8 * NT - 1) / (8 * NT);
  // blocks per row tile: enough that every SM has a few, at least one chunk a warp
  int S = 1;
  while (S < 8 && tiles * tt * S < 2 * sm_count() && a.w.nc >= (int64_t)2 * S * kWarps) S *= 2;
  const int cols = (int)std::min<int64_t>(8 * NT, a.T);
  const int64_t most = (a.w.nc + S - 1) / S;
  int64_t slab = (kMaxXBytes / (uint32_t)(TERMS * cols) - 64) / 256;
  f.slab = (int)std::max<int64_t>(1, std::min<int64_t>(slab, most));
  const size_t smem = (size_t)qm::x_pitch(f.slab) * TERMS * cols;
  static std::atomic<unsigned long long> done;
  cudaError_t e = ensure_smem_limit((const void*)k, kMaxXBytes, done);
  if (e != cudaSuccess) return e;
  for (int64_t y0 = 0; y0 < tt; y0 += 65535) {   // grid.y limit
    FewArgs g = f;
    g.x = static_cast<const TX*>(a.x) + y0 * 8 * NT * a.w.n;
    g.y = static_cast<TX*>(a.y) + y0 * 8 * NT * a.w.m;
    g.T = a.T - y0 * 8 * NT;
    g.vec_ok = aligned_to(g.x, 16) && (a.w.n * sizeof(TX)) % 16 == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * S), (unsigned)std::min<int64_t>(65535, tt - y0), 1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    count_launch();
    e = cudaLaunchKernelEx(&cfg, k, g);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename TX, typename H, int TERMS>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  const bool wide = a.w.ng == 1 || a.w.g % 128 == 0;
  if (a.T <= 8) return wide ? run<TX, H, TERMS, 1, 1, 1>(a, s) : run<TX, H, TERMS, 1, 1, 4>(a, s);
  return wide ? run<TX, H, TERMS, 2, 1, 1>(a, s) : run<TX, H, TERMS, 2, 1, 4>(a, s);
}

}  // namespace

cudaError_t launch_linear_few(const LinearArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case BAKRON_F32: return pick<float, __nv_bfloat16, 3>(a, s);
    case BAKRON_BF16: return pick<__nv_bfloat16, __nv_bfloat16, 1>(a, s);
    default: return pick<__half, __half, 1>(a, s);
  }
}

}  // namespace bakron
