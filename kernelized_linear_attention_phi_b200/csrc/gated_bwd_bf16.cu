// Gated linear attention, gradients, bf16 (gated_bwd.cuh).

#include "gated_bwd.cuh"

namespace la {

template cudaError_t gated_bwd_q_t<__nv_bfloat16>(
    const Problem&, const void*, const void*, const void*, const uint8_t*, const void*, const float*, int, int, void*, float*,
    float*, float*, float*, void*, cudaStream_t);
template cudaError_t gated_bwd_kv_t<__nv_bfloat16>(
    const Problem&, const void*, const void*, const void*, const void*, const uint8_t*, const void*, const float*, int, int,
    const float*, const float*, const float*, const float*, const void*, void*, void*, void*, cudaStream_t);

}  // namespace la
