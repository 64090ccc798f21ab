// Gated linear attention, forward, fp32 (gated_fwd.cuh).

#include "gated_fwd.cuh"

namespace la {

template cudaError_t gated_sweep_t<float>(
    const Problem&, const void*, const void*, const void*, const uint8_t*, const float*, const float*, const float*, int, int,
    void*, float*, float*, cudaStream_t);
template cudaError_t gated_states_t<float>(
    const Problem&, bool, const void*, const void*, const uint8_t*, const float*, const float*, int, int, int, int, bool, float*,
    float*, cudaStream_t);

}  // namespace la
