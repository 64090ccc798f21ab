// Norm of queries and keys with the position rotation (qk_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <la.h>

namespace la {

cudaError_t qk_norm_rope(const la_rope_desc& p, const void* q, const la_strides& qs, const void* k, const la_strides& ks,
                         const float* wq, const float* wk, const float* cos, const float* sin, const int32_t* positions,
                         void* q_out, void* k_out, cudaStream_t st);
// part: qk_rope_partials(p) rows of d floats for the weights' gradients.
cudaError_t qk_norm_rope_backward(const la_rope_desc& p, const void* q, const la_strides& qs, const void* k,
                                  const la_strides& ks, const float* wq, const float* wk, const float* cos,
                                  const float* sin, const int32_t* positions, const void* dq_out, const void* dk_out,
                                  void* dq, const la_strides& dqs, void* dk, const la_strides& dks, float* dwq, float* dwk,
                                  float* part, cudaStream_t st);
// Partial rows the backward pass writes for a device of `sms` SMs.
size_t qk_rope_partials(const la_rope_desc& p, int sms);

}  // namespace la
