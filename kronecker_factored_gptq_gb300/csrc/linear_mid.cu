// bakron_linear for some tens of tokens: Y = X V^T with up to 64 rows of X (16 of
// fp32, which count three times).
//
// Each code still meets few enough tokens that its bytes count (m n / 2), but
// now the activations, read again by every block of rows, would be more than
// that if each block were small.  So a block takes 16 rows per warp, up to 256,
// and all its warps walk through the columns together, 256 at a time, on
// activations that the block copies into shared memory; its codes go the way
// of the few-token kernel (qmma.cuh).  Both are asynchronous copies a few
// steps ahead, one barrier a step.  The matrix instructions of 8 tokens each are the
// next bound: 8 NT per 16 x 128 codes, each about 16 cycles of an SM's quarter.
// Measured: 32 tokens of 8192 x 8192 bf16 24 us, 48 of 14336 x 4096 fp16 with groups of
// 64 33 us (the codes' bytes alone: 5.4 us).
//
// Warps per block W and blocks per row group S (a cluster that splits the columns
// and adds the sums in rank order through distributed shared memory) are chosen
// to fill the SMs in one round where that can be; how many clusters fit at once
// is asked of the runtime.
#include <cooperative_groups.h>

#include <algorithm>

#include "linear.cuh"
#include "qmma.cuh"

namespace bakron {

namespace cg = cooperative_groups;

namespace {

constexpr int kMaxWarps = 16;
constexpr int kDepth = 3;                    // steps of 256 columns in flight, and at hand
constexpr uint32_t kPitch = 512 + 64;        // of a token's 256 columns: banks differ from row to row

struct MidArgs {
  PackedView w;
  const void* x;      // T rows of ld 16-bit values, 16-byte aligned
  void* y;
  int64_t ld;
  int cols;           // columns of x that exist, a multiple of 8
  int T, S, terms_plane;   // rows between the terms of x
};

template <typename TO, typename H, int TERMS, int NT, int NS>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) linear_mid_kernel(const __grid_constant__ MidArgs a) {
  using P = qm::Pipe<1, NS, kDepth>;
  extern __shared__ __align__(16) uint8_t dsm[];
  const int warps = blockDim.x >> 5;
  const int S = a.S, rank = S > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block_rows = 16 * warps;
  const int64_t row0 = (int64_t)(blockIdx.x / S) * block_rows;
  const int64_t rows[1] = {row0 + 16 * warp};
  const int nc = (int)a.w.nc, np = (nc + 1) / 2;
  const int p0 = np * rank / S, p1 = np * (rank + 1) / S;
  const int c_hi = min(nc, 2 * p1);

  qm::TileRef<1> tile;
  qm::tile_ref<1>(tile, a.w, 0, rows, lane);
  P pipe;
  pipe.base = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warp * P::kBytes;
  // activations: slots [term][token][256 columns]
  const uint32_t xs = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warps * P::kBytes;
  const uint32_t plane = (uint32_t)a.T * kPitch, slot_bytes = TERMS * plane;
  uint32_t fill = 0, read = 0;
  int ahead = p0;
  auto issue = [&]() {
    if (ahead < p1) {
      const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)ahead * 256;
      const int piece = threadIdx.x & 31;
      const uint32_t there = ahead * 256 + piece * 8 < a.cols ? 16u : 0u;    // zeros past the columns
      for (int i = warp; i < TERMS * a.T; i += warps) {
        const int q = TERMS == 1 ? 0 : i / a.T, t = i - q * a.T;
        const uint16_t* src = x + ((int64_t)q * a.terms_plane + t) * a.ld + (there ? piece * 8 : 0);
        if (!there) src = static_cast<const uint16_t*>(a.x);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(xs + fill + q * plane + t * kPitch + piece * 16),
                     "l"(src), "r"(there)
                     : "memory");
      }
    }
    pipe.issue(a.w, tile, 2 * ahead, ahead < p1 ? min(2, c_hi - 2 * ahead) : 0, lane);
    ++ahead;
    fill = fill + slot_bytes == kDepth * slot_bytes ? 0 : fill + slot_bytes;
  };
  if (2 * ahead + 1 < c_hi) qm::prefetch_codes<1>(tile, 2 * ahead, lane);
  grid_dep_wait();
  grid_dep_launch();
#pragma unroll
  for (int p = 0; p < kDepth - 1; ++p) issue();

  uint32_t col[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    col[j] = xs + (uint32_t)min(8 * j + (lane >> 2), a.T - 1) * kPitch + (uint32_t)(lane & 3) * 16;
  float tot[1][NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) tot[0][j][i] = 0.f;
  uint32_t z[1][2][NS];
  qm::load_zeros<1, NS>(z, a.w, tile, 2 * p0);
  for (int p = p0; p < p1; ++p) {
    // the slot that is filled now was read in the step before
    __syncthreads();
    issue();
    pipe.wait();
    __syncthreads();        // every thread's copies of this step have landed
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 2 * p + h;
      if (c < c_hi) {
        qm::Chunk16<NS> f[1];
        pipe.take(f, h, lane);
        qm::set_zeros<1, NS>(f, z);
        if (c + 1 < c_hi) qm::load_zeros<1, NS>(z, a.w, tile, c + 1);
        const uint32_t at = read + h * 256;
        qm::chunk_product<H, TERMS, 1, NT, NS>(
            tot, f, a.w.zero != nullptr, a.w.zu,
            [&](int j, int q, int s) { return qm::lds128(col[j] + q * plane + at + s * 64); });
      }
    }
    pipe.release();
    read = read + slot_bytes == kDepth * slot_bytes ? 0 : read + slot_bytes;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

  TO* y = static_cast<TO*>(a.y) + row0;
  if (S == 1) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 8 * j + 2 * (lane & 3) + (i & 1), r = 16 * warp + (lane >> 2) + 8 * (i >> 1);
        if (t < a.T && row0 + r < a.w.m) y[(int64_t)t * a.w.m + r] = from_float<TO>(tot[0][j][i]);
      }
    return;
  }
  // the blocks' sums [token][row], in the place of the copies
  __syncthreads();
  float* part = reinterpret_cast<float*>(dsm);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * j + 2 * (lane & 3) + (i & 1), r = 16 * warp + (lane >> 2) + 8 * (i >> 1);
      if (t < a.T) part[t * block_rows + r] = tot[0][j][i];
    }
  cg::cluster_group cluster = cg::this_cluster();
  __syncwarp();
  cluster.sync();
  for (int i = rank * (int)blockDim.x + threadIdx.x; i < a.T * block_rows; i += S * (int)blockDim.x) {
    const int t = i / block_rows, r = i - t * block_rows;
    float v = 0.f;
    for (int k = 0; k < S; ++k) v += cluster.map_shared_rank(part, k)[i];
    if (row0 + r < a.w.m) y[(int64_t)t * a.w.m + r] = from_float<TO>(v);
  }
  __syncwarp();
  cluster.sync();   // no block leaves while its sums are read
}

constexpr size_t kSmem = 226 * 1024;

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  Launch() = default;
  Launch(const Launch& o) : cfg(o.cfg) {
    at[0] = o.at[0];
    at[1] = o.at[1];
    cfg.attrs = at;
  }
};

Launch cluster_config(int threads, size_t smem, int cluster, unsigned blocks, cudaStream_t s) {
  Launch q;
  q.cfg.gridDim = dim3(blocks);
  q.cfg.blockDim = dim3((unsigned)threads);
  q.cfg.dynamicSmemBytes = smem;
  q.cfg.stream = s;
  q.at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  q.at[0].val.programmaticStreamSerializationAllowed = 1;
  q.at[1].id = cudaLaunchAttributeClusterDimension;
  q.at[1].val.clusterDim.x = (unsigned)cluster;
  q.at[1].val.clusterDim.y = q.at[1].val.clusterDim.z = 1;
  q.cfg.attrs = q.at;
  q.cfg.numAttrs = cluster > 1 ? 2 : 1;
  return q;
}

template <typename TO, typename H, int TERMS, int NT, int NS>
cudaError_t run(const LinearArgs& a, cudaStream_t s) {
  auto k = linear_mid_kernel<TO, H, TERMS, NT, NS>;
  MidArgs f = {};
  f.w = a.w;
  f.x = a.x;
  f.y = a.y;
  f.T = (int)a.T;
  f.ld = a.w.n;
  f.cols = (int)a.w.n;
  f.terms_plane = (int)a.T;
  if (TERMS != 1 || !aligned_to(a.x, 16) || a.w.n % 8 != 0) {
    const int64_t kp = a.w.nc * 128;
    const cudaError_t e = launch_planes(a.x, a.dtype, a.T, a.w.n, kp, a.ws, s);
    if (e != cudaSuccess) return e;
    f.x = a.ws;
    f.ld = kp;
    f.cols = (int)kp;
  }
  static_assert(8 * qm::Pipe<1, NS, kDepth>::kBytes + (size_t)kDepth * TERMS * 8 * NT * kPitch <= kSmem);
  static std::atomic<unsigned long long> done;
  cudaError_t e = ensure_smem_limit((const void*)k, kSmem, done);
  if (e != cudaSuccess) return e;
  // Warps per block and blocks per row group: the least time in units of a
  // 256-column step of 16 warps, a quarter of which a step costs whatever its
  // warps, and 8 of which a round of blocks costs to start and to join.
  const int64_t tiles = a.w.mp / 16, np = (a.w.nc + 1) / 2;
  auto ring = [&](int w) {
    return (size_t)w * qm::Pipe<1, NS, kDepth>::kBytes + (size_t)kDepth * TERMS * a.T * kPitch;
  };
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  int warps = 8, S = 1;      // whose memory always fits
  double best = 0.0;
  for (int c = 1; c <= 8 && c <= np; c *= 2) {
    // row groups at once on each device, by c = 1, 2, 4, 8 (0: not asked yet)
    static std::atomic<int> fit[64][4];
    std::atomic<int>* const kept = dev < 64 ? &fit[dev][c == 8 ? 3 : c / 2] : nullptr;
    int at_once = kept ? kept->load(std::memory_order_relaxed) : 0;
    if (at_once == 0) {
      at_once = sm_count();
      if (c > 1) {
        Launch q = cluster_config(32 * kMaxWarps, kSmem, c, c, s);
        e = cudaOccupancyMaxActiveClusters(&at_once, k, &q.cfg);
        if (e != cudaSuccess) return e;
      }
      if (at_once < 1) at_once = 1;
      if (kept) kept->store(at_once, std::memory_order_relaxed);
    }
    for (int w = kMaxWarps; w >= 8; --w) {
      if (ring(w) > kSmem) continue;
      const int64_t groups = (tiles + w - 1) / w;
      const double rounds = (double)((groups + at_once - 1) / at_once);
      const double cost = rounds * ((double)((np + c - 1) / c) * (w / 16.0 + 0.25) + 8.0);
      if (best == 0.0 || cost < best) {
        best = cost;
        warps = w;
        S = c;
      }
    }
  }
  f.S = S;
  const size_t smem = std::max<size_t>(ring(warps), S > 1 ? (size_t)a.T * 16 * warps * 4 : 0);
  Launch q = cluster_config(32 * warps, smem, S, (unsigned)((tiles + warps - 1) / warps * S), s);
  count_launch();
  return cudaLaunchKernelEx(&q.cfg, k, f);
}

template <typename TO, int NT>
cudaError_t by_groups(const LinearArgs& a, cudaStream_t s) {
  const bool wide = a.w.ng == 1 || a.w.g % 128 == 0;
  return wide ? run<TO, TO, 1, NT, 1>(a, s) : run<TO, TO, 1, NT, 4>(a, s);
}

template <typename TO>
cudaError_t by_tokens(const LinearArgs& a, cudaStream_t s) {
  if (a.T <= 16) return by_groups<TO, 2>(a, s);
  if (a.T <= 32) return by_groups<TO, 4>(a, s);
  if (a.T <= 48) return by_groups<TO, 6>(a, s);
  return by_groups<TO, 8>(a, s);
}

}  // namespace

cudaError_t launch_linear_mid(const LinearArgs& a, cudaStream_t s) {
  if (a.dtype == BAKRON_F32) {
    const bool wide = a.w.ng == 1 || a.w.g % 128 == 0;
    if (a.T <= 8)
      return wide ? run<float, __nv_bfloat16, 3, 1, 1>(a, s) : run<float, __nv_bfloat16, 3, 1, 4>(a, s);
    return wide ? run<float, __nv_bfloat16, 3, 2, 1>(a, s) : run<float, __nv_bfloat16, 3, 2, 4>(a, s);
  }
  return a.dtype == BAKRON_BF16 ? by_tokens<__nv_bfloat16>(a, s) : by_tokens<__half>(a, s);
}

}  // namespace bakron
