// bakron_linear_act for up to 16 tokens.
#include "linear_few.cuh"

namespace bakron {

cudaError_t launch_linear_act_few(const LinearArgs& a, cudaStream_t s) { return few<true>(a, s); }

}  // namespace bakron
