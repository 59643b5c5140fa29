// bakron_linear for some tens of tokens.
#include "linear_mid.cuh"

namespace bakron {

cudaError_t launch_linear_mid(const LinearArgs& a, cudaStream_t s) { return mid<false>(a, s); }

}  // namespace bakron
