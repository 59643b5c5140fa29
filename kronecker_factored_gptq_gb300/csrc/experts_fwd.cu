// bakron_experts.
#include "linear_fwd.cuh"

namespace bakron {

cudaError_t launch_experts_fwd(const LinearArgs& a, cudaStream_t s) { return forward<kExperts>(a, s); }

}  // namespace bakron
