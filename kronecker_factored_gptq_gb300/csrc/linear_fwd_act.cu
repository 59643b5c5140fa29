// bakron_linear_act for many tokens.
#include "linear_fwd.cuh"

namespace bakron {

cudaError_t launch_linear_act_fwd(const LinearArgs& a, cudaStream_t s) { return forward<kWithAct>(a, s); }

}  // namespace bakron
