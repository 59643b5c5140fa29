// bakron_linear for up to 16 tokens.
#include "linear_few.cuh"

namespace bakron {

cudaError_t launch_linear_few(const LinearArgs& a, cudaStream_t s) { return few<false>(a, s); }

}  // namespace bakron
