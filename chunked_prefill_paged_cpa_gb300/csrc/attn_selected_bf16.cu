// The step kernel over selected pages, for bf16 queries and caches.
#include "attn_step.cuh"

namespace cpa {
template cudaError_t launch_step<0, kSelected>(const AttnParams &, const StepWs &, cudaStream_t);
}  // namespace cpa
