// bakron_linear_act for some tens of tokens.
#include "linear_mid.cuh"

namespace bakron {

cudaError_t launch_linear_act_mid(const LinearArgs& a, cudaStream_t s) { return mid<true>(a, s); }

}  // namespace bakron
