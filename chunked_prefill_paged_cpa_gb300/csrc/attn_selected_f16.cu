// The step kernel over selected pages, for binary16 queries and caches.
#include "attn_step.cuh"

namespace cpa {
template cudaError_t launch_step<1, kSelected>(const AttnParams &, const StepWs &, cudaStream_t);
}  // namespace cpa
