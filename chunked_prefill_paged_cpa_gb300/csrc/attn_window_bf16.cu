// The step kernel with a sliding window and sinks, for bf16 queries and caches.
#include "attn_step.cuh"

namespace cpa {
template cudaError_t launch_step<0, true>(const AttnParams &, const StepWs &, cudaStream_t);
}  // namespace cpa
