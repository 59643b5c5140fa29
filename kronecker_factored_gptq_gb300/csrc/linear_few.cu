// bakron_linear for up to 16 tokens: Y = X V^T.
//
// y_ti = sum_k s_ik sum_{j in group k} x_tj (u_ij - z_ik).  Each code is read
// once and used for at most 16 tokens, so the codes' bytes bound the kernel
// (m n / 2; at 8192 x 8192 33.6 MB, 5.0 us at 6.68 TB/s); the products run on
// warp-level matrix instructions (qmma.cuh), which cost a fraction of that.  Measured:
// 1 token of 8192 x 8192 bf16 10.4 us (3.3 TB/s), 16 tokens 16 us; 1 token of 1024 x 1024
// 1.8 us and 7 of 1000 x 1111 fp32 4.3 us, which are launch and latency.  What bounds
// the large ones is the latency of a warp's dependent instructions (some 350 per 32 x 128
// codes): 44 % of the issue slots and a fifth of the warps an SM could hold are in use.
//
// A block takes 16 or 32 rows; its 8 warps take the 128-column chunks of the rows in
// turn, each with several chunks on their way, and add their partial sums in
// shared memory in a fixed order.  An activation meets one warp of a block only,
// so 16-bit activations are read where they are; fp32 ones (which become three
// terms) and rows that are not 16-byte aligned are staged in shared memory.  Few
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
constexpr uint32_t kMaxXBytes = 64 * 1024;   // activations staged at a time

struct FewArgs {
  PackedView w;
  const void* x;
  void* y;
  int64_t T;
  int S;         // blocks per row tile (a cluster)
  int slab;      // chunks of activations staged at a time; 0: read in place
  int vec_ok;    // rows of x are 16-byte aligned
};

// Slots of two chunks per warp.
template <int RT>
constexpr int kDepth = RT == 1 ? 3 : 2;

template <typename TX, typename H, int TERMS, int NT, int RT, int NS>
__global__ void __launch_bounds__(kThreads, 2) linear_few_kernel(const __grid_constant__ FewArgs a) {
  using P = qm::Pipe<RT, NS, kDepth<RT>>;
  constexpr int ROWS = 16 * RT, OUT = NT * 8 * ROWS;
  extern __shared__ __align__(16) uint8_t dsm[];      // the warps' chunks, then staged activations
  __shared__ float red[kWarps][NT * 8][ROWS];
  __shared__ float part[OUT];
  const int S = a.S, rank = S > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)(blockIdx.x / S) * ROWS;
  int64_t rows[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) rows[r] = row0 + 16 * r;
  const int t0 = blockIdx.y * (8 * NT);
  const int cols = min(8 * NT, (int)a.T - t0);
  const TX* x = static_cast<const TX*>(a.x) + t0 * a.w.n;
  const int nc = (int)a.w.nc;
  const int c_lo = nc * rank / S, c_hi = nc * (rank + 1) / S;

  qm::TileRef<RT> tile;
  qm::tile_ref<RT>(tile, a.w, 0, rows, lane);
  P pipe;
  pipe.base = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warp * P::kBytes;
  // the warps take the chunks two by two, in turn
  int ahead = c_lo + 2 * warp;
  if (ahead + 1 < c_hi) qm::prefetch_codes<RT>(tile, ahead, lane);
  grid_dep_wait();
  grid_dep_launch();
  auto issue = [&]() {
    pipe.issue(a.w, tile, ahead, max(0, min(2, c_hi - ahead)), lane);
    ahead += 2 * kWarps;
  };
#pragma unroll
  for (int p = 0; p < kDepth<RT> - 1; ++p) issue();

  int col[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) col[j] = min(8 * j + (lane >> 2), cols - 1);
  float tot[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[r][j][i] = 0.f;

  uint32_t z[RT][2][NS];
  if (c_lo + 2 * warp < c_hi) qm::load_zeros<RT, NS>(z, a.w, tile, c_lo + 2 * warp);
  qm::Chunk16<NS> f[RT];
  // chunk c, half h of the slot at hand; its successor's zero points are on their way
  auto half = [&](int c, int h, auto fetch) {
    pipe.take(f, h, lane);
    qm::set_zeros<RT, NS>(f, z);
    const int next = h == 0 && c + 1 < c_hi ? c + 1 : c - h + 2 * kWarps;
    if (next < c_hi) qm::load_zeros<RT, NS>(z, a.w, tile, next);
    qm::chunk_product<H, TERMS, RT, NT, NS>(tot, f, a.w.zero != nullptr, a.w.zu, fetch);
  };
  if (TERMS == 1 && a.slab == 0) {
    const TX* xr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xr[j] = x + (int64_t)col[j] * a.w.n + 8 * (lane & 3);
    const int whole = (int)(a.w.n / 128);       // chunks without padding
    for (int c = c_lo + 2 * warp; c < c_hi; c += 2 * kWarps) {
      issue();
      pipe.wait();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (c + h < min(whole, c_hi)) {
          half(c + h, h, [&](int j, int, int s) {
            return __ldg(reinterpret_cast<const uint4*>(xr[j] + (c + h) * 128 + 32 * s));
          });
        } else if (c + h < c_hi) {
          half(c + h, h, [&](int j, int, int s) {
            const int k = (c + h) * 128 + 32 * s;
            return k + 8 * (lane & 3) < a.w.n ? __ldg(reinterpret_cast<const uint4*>(xr[j] + k))
                                              : make_uint4(0, 0, 0, 0);
          });
        }
      }
      pipe.release();
    }
  } else {
    uint8_t* xs = dsm + kWarps * P::kBytes;
    const uint32_t pitch = qm::x_pitch(a.slab);      // slab is even
    const uint32_t plane = pitch * (uint32_t)cols;
    int c = c_lo + 2 * warp;
    for (int s0 = c_lo; s0 < c_hi; s0 += a.slab) {
      const int s1 = min(s0 + a.slab, c_hi);
      if (s0 != c_lo) __syncthreads();
      qm::stage_x<TX, TERMS>(xs, plane, pitch, x, a.w.n, cols, [](int r) { return (int64_t)r; }, s0 * 128,
                             s1 - s0, a.w.n, a.vec_ok != 0);
      __syncthreads();
      for (; c < s1; c += 2 * kWarps) {
        issue();
        pipe.wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (c + h < s1) {
            const uint8_t* xc = xs + (c + h - s0) * 256 + (lane & 3) * 16;
            half(c + h, h, [&](int j, int q, int s) {
              return *reinterpret_cast<const uint4*>(xc + q * plane + (uint32_t)col[j] * pitch + s * 64);
            });
          }
        }
        pipe.release();
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  // partial sums of the warps: [column][row], rows fastest
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int o = 16 * r + (lane >> 2), c = 8 * j + 2 * (lane & 3);
      red[warp][c][o] = tot[r][j][0];
      red[warp][c + 1][o] = tot[r][j][1];
      red[warp][c][o + 8] = tot[r][j][2];
      red[warp][c + 1][o + 8] = tot[r][j][3];
    }
  __syncthreads();
  TX* y = static_cast<TX*>(a.y) + t0 * a.w.m + row0;
  for (int i = threadIdx.x; i < OUT; i += kThreads) {
    const int c = i / ROWS, r = i % ROWS;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][c][r];
    if (S > 1) part[i] = v;
    else if (c < cols && row0 + r < a.w.m) y[c * a.w.m + r] = from_float<TX>(v);
  }
  if (S > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    __syncwarp();
    cluster.sync();
    if (rank == 0) {
      for (int i = threadIdx.x; i < OUT; i += kThreads) {
        const int c = i / ROWS, r = i % ROWS;
        if (c >= cols || row0 + r >= a.w.m) continue;
        float v = 0.f;
        for (int k = 0; k < S; ++k) v += cluster.map_shared_rank(part, k)[i];
        y[c * a.w.m + r] = from_float<TX>(v);
      }
    }
    __syncwarp();
    cluster.sync();   // no block leaves while its sums are read
  }
}

template <typename TX, typename H, int TERMS, int NT, int RT, int NS>
cudaError_t run(const LinearArgs& a, cudaStream_t s) {
  auto k = linear_few_kernel<TX, H, TERMS, NT, RT, NS>;
  constexpr size_t ring = kWarps * qm::Pipe<RT, NS, kDepth<RT>>::kBytes;
  FewArgs f;
  f.w = a.w;
  f.x = a.x;
  f.y = a.y;
  f.T = a.T;
  f.vec_ok = aligned_to(a.x, 16) && (a.w.n * sizeof(TX)) % 16 == 0;
  const int64_t tiles = (a.w.mp + 16 * RT - 1) / (16 * RT);
  const int64_t tt = (a.T + 8 * NT - 1) / (8 * NT);   // T <= kFewTokens: a handful
  // blocks per row tile: enough that every SM has one or two, at least one slot
  // a warp
  f.S = 1;
  while (f.S < 8 && tiles * tt * f.S < sm_count() && a.w.nc >= (int64_t)2 * f.S * kWarps) f.S *= 2;
  size_t smem = ring;
  f.slab = 0;
  if (TERMS != 1 || !f.vec_ok) {
    const int cols = (int)std::min<int64_t>(8 * NT, a.T);
    const int64_t slab = (kMaxXBytes / (uint32_t)(TERMS * cols) - 64) / 256;
    f.slab = (int)std::max<int64_t>(2, std::min<int64_t>(slab, (a.w.nc + f.S - 1) / f.S + 1) / 2 * 2);
    smem += (size_t)qm::x_pitch(f.slab) * TERMS * cols;
  }
  static std::atomic<unsigned long long> done;
  cudaError_t e = ensure_smem_limit((const void*)k, ring + kMaxXBytes, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * f.S), (unsigned)tt, 1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)f.S;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = f.S > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, k, f);
}

template <typename TX, typename H, int TERMS, int NT, int NS>
cudaError_t by_rows(const LinearArgs& a, cudaStream_t s) {
  // two row tiles a warp once that leaves a block for every SM
  return a.w.mp >= (int64_t)32 * sm_count() ? run<TX, H, TERMS, NT, 2, NS>(a, s) : run<TX, H, TERMS, NT, 1, NS>(a, s);
}

template <typename TX, typename H, int TERMS>
cudaError_t pick(const LinearArgs& a, cudaStream_t s) {
  const bool wide = a.w.ng == 1 || a.w.g % 128 == 0;
  if (a.T <= 8) return wide ? by_rows<TX, H, TERMS, 1, 1>(a, s) : by_rows<TX, H, TERMS, 1, 4>(a, s);
  return wide ? by_rows<TX, H, TERMS, 2, 1>(a, s) : by_rows<TX, H, TERMS, 2, 4>(a, s);
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
