// bakron_linear for many tokens.
#include "linear_fwd.cuh"

namespace bakron {

// Of any of its kernels: each has an SM to itself.
int linear_fwd_eights() {
  static std::atomic<int> kept[64];          // by device, one more than the number
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  n = kept[dev].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  auto k = linear_fwd_kernel<__nv_bfloat16, __nv_bfloat16, 1, 96, 8, 8, 1, kPlain>;
  constexpr size_t smem = kRing + kCodes + 1024;
  static std::atomic<unsigned long long> done;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 8;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(8);
  cfg.blockDim = dim3(32 * 20);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (ensure_smem_limit((const void*)k, smem, done) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 0) {
    (void)cudaGetLastError();
    n = 0;
  }
  kept[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

int64_t linear_fwd_steps(const LinearArgs& a) {
  const int N = cut_of(a).N;
  const int64_t tiles = (a.w.m + 127) / 128 * ((a.T + N - 1) / N);
  const int S = blocks_per_tile(tiles, a.w.nc);
  return S > 1 ? (a.w.nc + S - 1) / S : (tiles + sm_count() - 1) / sm_count() * a.w.nc;
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t s) { return forward<kPlain>(a, s); }

}  // namespace bakron
