// bakron_linear_grad.
#include "linear_grad.cuh"

namespace bakron {

cudaError_t launch_linear_grad(const LinearArgs& a, cudaStream_t s) { return gradient<kPlain>(a, s); }

}  // namespace bakron
