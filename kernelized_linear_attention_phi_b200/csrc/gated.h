// Gated linear attention: kernels behind la_gated_causal,
// la_gated_causal_backward and la_gated_decode_step.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"

namespace la {

// Records of all chunks' gates, gated_gate_bytes(p) bytes, which the calls below
// take in the place of g.
cudaError_t gated_gates(const Problem& p, const void* g, uint8_t* out, cudaStream_t st);
size_t gated_gate_bytes(const Problem& p);
// Outputs (not bf16 at d = 128: tc_gated_sweep) of every block of block_tokens tokens (a multiple of 64) from the
// state in front of it: record (bh, blk) of `prefix`, or with prefix null (one
// block) S_in / z_in, or zero. S_out / z_out (one block only): the state after
// the last token.
cudaError_t gated_sweep(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const float* prefix,
                        const float* S_in, const float* z_in, int block_tokens, int nblk, void* out, float* S_out,
                        float* z_out, cudaStream_t st);
// Own states of `count` blocks from blk0 on: records rec[bh*nblk + blk] and the
// products of the blocks' gates dec[bh*nblk + blk]. Forward: x = k, y = v, up,
// col null. Reverse (gradients): x = q, y = dout; up, col as the first sweep
// left them, null when not normalized. exact: the terms of the
// states keep all their bits (bf16), for a state that goes to the caller.
cudaError_t gated_states(const Problem& p, bool reverse, const void* x, const void* y, const uint8_t* gates, const float* up,
                         const float* col, int block_tokens, int nblk, int blk0, int count, bool exact, float* rec, float* dec,
                         cudaStream_t st);
// In place: record blk becomes the state in front of block blk (reverse:
// behind it). S_out / z_out (may be null, may alias S_in / z_in): the state
// past the last (reverse: first) block; without them that block's own record
// is not read.
cudaError_t gated_scan(const Problem& p, bool reverse, float* rec, const float* dec, int nblk, const float* S_in,
                       const float* z_in, float* S_out, float* z_out, cudaStream_t st);
// The same on tcgen05 tensor cores (tc_gated.cu): bf16, d = 128, states and
// outputs, from g itself (reverse states: up and col, null when not normalized).
// An expired wait sets tc::FLAG_TIMEOUT in *err.
bool tc_gated_supported(const Problem& p);
cudaError_t tc_gated_states(const Problem& p, bool reverse, const void* x, const void* y, const void* g, const float* up,
                            const float* col, int block_tokens, int nblk, int blk0, int count, bool exact, float* part,
                            float* dec, uint32_t* err, cudaStream_t st);
cudaError_t tc_gated_sweep(const Problem& p, const void* q, const void* k, const void* v, const void* g,
                           const float* prefix, const float* S_in, const float* z_in, int block_tokens, int nblk, void* out,
                           uint32_t* err, cudaStream_t st);

// One token: S_out = e^g S + phi(k) (x) v and so on, read out. S_out / z_out
// may be S / z.
cudaError_t gated_decode(const Problem& p, const void* q, const void* k, const void* v, const void* g, const float* S,
                         const float* z, float* S_out, float* z_out, void* out, cudaStream_t st);

// Gradients, first sweep (chunks in order): dq, and per token (normalized only)
// up = 1 / den, col = -(out . dout) and own = up (dout.v + col), the query's own
// key's; dgp (what the chunk's queries give to
// dg), and per chunk of gated_chunk(p) tokens the state in front of it
// (chunk_state, gated_chunk_state_bytes(p) each).
cudaError_t gated_bwd_q(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const void* dout,
                        const float* prefix, int block_tokens, int nblk, void* dq, float* up, float* col, float* own, float* dgp,
                        void* chunk_state, cudaStream_t st);
// Second sweep (chunks in reverse): dk, dv, dg from the states behind the blocks.
cudaError_t gated_bwd_kv(const Problem& p, const void* q, const void* k, const void* v, const void* g, const uint8_t* gates, const void* dout,
                         const float* suffix, int block_tokens, int nblk, const float* up, const float* col,
                         const float* own, const float* dgp, const void* chunk_state, void* dk, void* dv, void* dg, cudaStream_t st);
int gated_chunk(const Problem& p);
size_t gated_chunk_state_bytes(const Problem& p);

// The same per element type (gated_bf16.cu, gated_f32.cu, gated_bwd_bf16.cu, gated_bwd_f32.cu).
template <typename T>
cudaError_t gated_sweep_t(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const float* prefix,
                          const float* S_in, const float* z_in, int block_tokens, int nblk, void* out, float* S_out,
                          float* z_out, cudaStream_t st);
template <typename T>
cudaError_t gated_states_t(const Problem& p, bool reverse, const void* x, const void* y, const uint8_t* gates, const float* up,
                           const float* col, int block_tokens, int nblk, int blk0, int count, bool exact, float* rec, float* dec,
                           cudaStream_t st);
template <typename T>
cudaError_t gated_bwd_q_t(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const void* dout,
                          const float* prefix, int block_tokens, int nblk, void* dq, float* up, float* col, float* own, float* dgp,
                          void* chunk_state, cudaStream_t st);
template <typename T>
cudaError_t gated_bwd_kv_t(const Problem& p, const void* q, const void* k, const void* v, const void* g, const uint8_t* gates, const void* dout,
                           const float* suffix, int block_tokens, int nblk, const float* up, const float* col,
                           const float* own, const float* dgp, const void* chunk_state, void* dk, void* dv, void* dg, cudaStream_t st);

namespace gated {
// Calls f(integral_constant<D>, integral_constant<PHI>) for p.
template <typename F> cudaError_t dispatch(const Problem& p, F f) {
    auto with_phi = [&](auto d) -> cudaError_t {
        switch (p.phi) {
            case 0: return f(d, std::integral_constant<int, 0>{});
            case 1: return f(d, std::integral_constant<int, 1>{});
            case 2: return f(d, std::integral_constant<int, 2>{});
        }
        return cudaErrorInvalidValue;
    };
    switch (p.d) {
        case 16: return with_phi(std::integral_constant<int, 16>{});
        case 32: return with_phi(std::integral_constant<int, 32>{});
        case 64: return with_phi(std::integral_constant<int, 64>{});
        case 128: return with_phi(std::integral_constant<int, 128>{});
    }
    return cudaErrorInvalidValue;
}
}  // namespace gated

}  // namespace la
