// bakron_linear for many tokens.
#include "linear_fwd.cuh"

namespace bakron {

int64_t linear_fwd_steps(const LinearArgs& a) {
  const int N = tokens_per_tile(a, most_tokens(a), 32);
  const int64_t tiles = (a.w.m + 127) / 128 * ((a.T + N - 1) / N);
  const int S = blocks_per_tile(tiles, a.w.nc);
  return S > 1 ? (a.w.nc + S - 1) / S : (tiles + sm_count() - 1) / sm_count() * a.w.nc;
}

cudaError_t launch_linear_fwd(const LinearArgs& a, cudaStream_t s) { return forward<kPlain>(a, s); }

}  // namespace bakron
