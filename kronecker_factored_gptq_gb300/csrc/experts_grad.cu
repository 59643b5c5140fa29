// bakron_experts_grad.
#include "linear_grad.cuh"

namespace bakron {

cudaError_t launch_experts_grad(const LinearArgs& a, cudaStream_t s) { return gradient<kExperts>(a, s); }

}  // namespace bakron
