// Gated linear attention, forward (causal, with the decay a_t = exp(g_t)):
//   S_t = a_t S_{t-1} + phi(k_t) (x) v_t,  z_t = a_t z_{t-1} + phi(k_t),
//   out_t = phi(q_t) S_t / (phi(q_t) . z_t).
// Chunk by chunk, with b_i the log of the product of a chunk's gates up to i:
//   out_i = [ sum_{j <= i} e^{b_i - b_j} (phi(q_i).phi(k_j)) v_j + e^{b_i} phi(q_i) S ] / (the same with v = 1)
//   S    <- e^{b_last} S + sum_j e^{b_last - b_j} phi(k_j) (x) v_j
// e^{b_i - b_j} is taken as e^{b_i} e^{-b_j} where the chunk's sums allow it
// (gated_common.cuh, Gates).

#pragma once

#include "gated.h"
#include "gated_common.cuh"
#include "launch_util.h"

namespace la {
namespace gated {

template <typename T, int D> struct FwdSmem {
    using SH = Shape<T, D>;
    T tiles[SH::ST][3][SH::TILE];  // q, k, v
    T sop[SH::SB][SH::SOP];
    float zs[SH::SB][D];
    Gates<SH::C> gates[2];
};
template <typename T, int D> struct StateSmem {
    using SH = Shape<T, D>;
    T tiles[SH::ST][2][SH::TILE];
    Gates<SH::C> gates[2];
};

// The outputs of one block of a head's chunks, from the state in front of the
// block (a record of `prefix`, or S_in / z_in, or nothing). 4x16x8192x64 bf16:
// 109 us for 268 MB (2.5 TB/s; shared memory 68 % busy with operands, the tensor
// pipe 33 %, DRAM 29 %), fp32 451 us (three products for one). A short block is
// the latency of its chunks: 2x8x4096x64 in blocks of four chunks 19 us.
template <typename T, int D, int PHI>
__global__ void __launch_bounds__(Shape<T, D>::THREADS, D == 64 ? (sizeof(T) == 2 ? 4 : 3) : 1)
gated_sweep_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                   const uint8_t* __restrict__ gates, const float* prefix, const float* S_in, const float* z_in, int N, int block_tokens, int nblk,
                   int normalize, T* __restrict__ out, float* S_out, float* z_out) {
    using SH = Shape<T, D>;
    constexpr int C = SH::C, LD = SH::LD;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<FwdSmem<T, D>*>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    const int blk = blockIdx.x, bh = blockIdx.y;
    const int first = blk * block_tokens, end = min(N, first + block_tokens);
    const int nch = (end - first + C - 1) / C;
    const size_t off = (size_t)bh * N * D;
    q += off; k += off; v += off; out += off;
    gates += ((size_t)bh * ((N + C - 1) / C) + first / C) * kGateBytes<C>;
    pdl_wait();

    auto fetch = [&](int c) {
        const int row0 = first + c * C;
        load_gates<C>(sm.gates[c & 1], gates + (size_t)c * kGateBytes<C>, nullptr, nullptr, nullptr, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][0], q, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][1], k, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][2], v, row0, N);
        cp_async_commit();
    };
    fetch(0);
    State<T, D> st;
    if (prefix) {
        const float* rec = prefix + ((size_t)bh * nblk + blk) * (size_t)(D * D + D);
        st.seed(rec, rec + D * D, warp, lane);
    } else {
        st.seed(S_in ? S_in + (size_t)bh * D * D : nullptr, z_in ? z_in + (size_t)bh * D : nullptr, warp, lane);
    }
    st.publish(sm.sop[0], sm.zs[0], warp, lane);
    // the warps' row groups differ in work (a group sees the keys before it):
    // CTAs of an SM start them at different warps
    const int rg = row_group<SH>(warp), cg = warp / SH::RG;
    const int i0 = rg * 16, col0 = cg * SH::NCOL;

#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        cp_async_wait<0>();
        __syncthreads();
        if (SH::ST == 2 && c + 1 < nch) fetch(c + 1);
        const T *qt = sm.tiles[c % SH::ST][0], *kt = sm.tiles[c % SH::ST][1], *vt = sm.tiles[c % SH::ST][2];
        const Gates<C>& gs = sm.gates[c & 1];
        const int sb = SH::SB == 2 ? (c & 1) : 0;
        const T* sop = sm.sop[sb];
        const float* zs = sm.zs[sb];

        // The loop over the key groups stays rolled, in fp32 the channels' too: a
        // block often has only a few chunks, and then the time to fetch the code
        // counts (1x4x1531x32 fp32, elu + 1: 61 us unrolled, 23 rolled). bf16 gains
        // by the channels' products side by side (4x16x8192x64: 139 us -> 129).
        constexpr int NT = SH::NCOL / 8;
        float o[NT][4] = {}, oz[4] = {};
#pragma unroll(SH::F32 ? 1 : D / 16)
        for (int k0 = 0; k0 < D; k0 += 16) {
            FragA<T> a;
            load_a<LD>(a, qt, i0, k0, lane);
            phi_frag<PHI>(a);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                FragB<T> b[2];
                load_b<LD>(b, sop, k0, col0 + 16 * n, lane);
                mma_step(o[2 * n], a, b[0]);
                mma_step(o[2 * n + 1], a, b[1]);
            }
            if (normalize) {
                FragB<T> b;
                load_column(b, zs, k0, lane);
                mma_step(oz, a, b);
            }
        }
        const bool deep = gs.deep;
        const float f0 = gs.from_start[i0 + g], f1 = gs.from_start[i0 + g + 8];
        // z's product sits in columns 0 and 1 (t == 0); the row sums below add over the quad
        float den0 = t == 0 ? f0 * (oz[0] + oz[1]) : 0.f, den1 = t == 0 ? f1 * (oz[2] + oz[3]) : 0.f;
        const float hi0 = gs.hi[i0 + g], lo0 = gs.lo[i0 + g], hi1 = gs.hi[i0 + g + 8], lo1 = gs.lo[i0 + g + 8];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            o[n][0] *= f0; o[n][1] *= f0; o[n][2] *= f1; o[n][3] *= f1;
        }
#pragma unroll 1
        for (int jt = 0; jt <= rg; ++jt) {
            float p[2][4] = {};
#pragma unroll(SH::F32 ? 1 : D / 16)
            for (int k0 = 0; k0 < D; k0 += 16) {
                FragA<T> a;
                FragB<T> b[2];
                load_a<LD>(a, qt, i0, k0, lane);
                phi_frag<PHI>(a);
                load_bt<LD>(b, kt, jt * 16, k0, lane);
                phi_frag<PHI>(b[0]);
                phi_frag<PHI>(b[1]);
                mma_step(p[0], a, b[0]);
                mma_step(p[1], a, b[1]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int jl = n * 8 + 2 * t, j = jt * 16 + jl;
                if (deep) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[n][e] *= decay(gs, hi0, lo0, j + e);
                        p[n][2 + e] *= decay(gs, hi1, lo1, j + e);
                    }
                } else {
                    const float2 w = *reinterpret_cast<const float2*>(gs.inv + j);
                    p[n][0] *= f0 * w.x; p[n][1] *= f0 * w.y; p[n][2] *= f1 * w.x; p[n][3] *= f1 * w.y;
                }
                if (jt == rg) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (jl + e > g) p[n][e] = 0.f;
                        if (jl + e > g + 8) p[n][2 + e] = 0.f;
                    }
                }
            }
            // bf16: the weights are rounded once, as in the chunked forms without a
            // gate, and the denominator sums the rounded ones, so that the
            // output is a mean of the values with these very weights
            FragA<T> a;
            float w[8];
            make_a(a, p[0], p[1]);
            unpack(a, w);
            den0 += (w[0] + w[1]) + (w[4] + w[5]);
            den1 += (w[2] + w[3]) + (w[6] + w[7]);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                FragB<T> b[2];
                load_b<LD>(b, vt, jt * 16, col0 + 16 * n, lane);
                mma_step(o[2 * n], a, b[0]);
                mma_step(o[2 * n + 1], a, b[1]);
            }
        }
        float r0 = 1.f, r1 = 1.f;
        if (normalize) {
            r0 = 1.f / quad_sum(den0);
            r1 = 1.f / quad_sum(den1);
        }
        const int row = first + c * C + i0 + g;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            T* p = out + (size_t)row * D + col0 + 8 * n + 2 * t;
            if constexpr (SH::F32) {
                if (row < end) *reinterpret_cast<float2*>(p) = make_float2(o[n][0] * r0, o[n][1] * r0);
                if (row + 8 < end) *reinterpret_cast<float2*>(p + 8 * D) = make_float2(o[n][2] * r1, o[n][3] * r1);
            } else {
                if (row < end) *reinterpret_cast<uint32_t*>(p) = pack_bf16(o[n][0] * r0, o[n][1] * r0);
                if (row + 8 < end) *reinterpret_cast<uint32_t*>(p + 8 * D) = pack_bf16(o[n][2] * r1, o[n][3] * r1);
            }
        }
        if (c + 1 < nch || S_out) {
            st.template update<PHI>(kt, vt, gs.to_end, nullptr, nullptr, true, gs.all, warp, lane, S_out != nullptr);
            if (SH::SB == 1) __syncthreads();  // every warp has read the operand and the tiles
            if (c + 1 < nch) {
                if (SH::ST == 1) fetch(c + 1);
                const int nb = SH::SB == 2 ? ((c + 1) & 1) : 0;
                st.publish(sm.sop[nb], sm.zs[nb], warp, lane);
            }
        }
    }
    if (S_out) st.store(S_out + (size_t)bh * D * D, z_out + (size_t)bh * D, warp, lane);
}

// One block's own state (from zero) and the product of its gates. 4x16x8192x64
// bf16: 51 us for 134 MB, fp32 139 us.
//   REVERSE = false: X = k, Y = v, weights e^{b_last - b_j}, chunks in order;
//   REVERSE = true (gradients): X = q, Y = dout, weights e^{b_i} / den_i, the
//   z part weighted by col_i = -(out_i . dout_i), chunks from the last to the first.
template <typename T, int D, int PHI, bool REVERSE>
__global__ void __launch_bounds__(Shape<T, D>::THREADS)
gated_state_kernel(const T* __restrict__ x, const T* __restrict__ y, const uint8_t* __restrict__ gates,
                   const float* up, const float* col, int N, int block_tokens, int nblk, int blk0, bool exact,
                   float* __restrict__ rec, float* __restrict__ dec) {
    using SH = Shape<T, D>;
    constexpr int C = SH::C;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<StateSmem<T, D>*>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int blk = blk0 + blockIdx.x, bh = blockIdx.y;
    const int first = blk * block_tokens, end = min(N, first + block_tokens);
    const int nch = (end - first + C - 1) / C;
    x += (size_t)bh * N * D;
    y += (size_t)bh * N * D;
    gates += ((size_t)bh * ((N + C - 1) / C) + first / C) * kGateBytes<C>;
    if (up) {
        up += (size_t)bh * N;
        col += (size_t)bh * N;
    }
    pdl_wait();
    auto chunk = [&](int c) { return REVERSE ? nch - 1 - c : c; };
    auto fetch = [&](int c) {
        const int row0 = first + chunk(c) * C;
        load_gates<C>(sm.gates[c & 1], gates + (size_t)chunk(c) * kGateBytes<C>, up, col, nullptr, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][0], x, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][1], y, row0, N);
        cp_async_commit();
    };
    fetch(0);
    State<T, D> st;
    st.seed(nullptr, nullptr, warp, lane);
    float total = 1.f;
#pragma unroll 1
    for (int c = 0; c < nch; ++c) {
        cp_async_wait<0>();
        __syncthreads();
        if (SH::ST == 2 && c + 1 < nch) fetch(c + 1);
        const Gates<C>& gs = sm.gates[c & 1];
        st.template update<PHI>(sm.tiles[c % SH::ST][0], sm.tiles[c % SH::ST][1], REVERSE ? gs.from_start : gs.to_end,
                                REVERSE && up ? gs.up : nullptr, REVERSE ? gs.col : nullptr, !REVERSE || up, gs.all, warp, lane, !REVERSE && exact);
        total *= gs.all;
        if (SH::ST == 1 && c + 1 < nch) {
            __syncthreads();  // every warp has read the tiles
            fetch(c + 1);
        }
    }
    float* r = rec + ((size_t)bh * nblk + blk) * (size_t)(D * D + D);
    st.store(r, r + D * D, warp, lane);
    if (threadIdx.x == 0) dec[(size_t)bh * nblk + blk] = total;
}

template <typename T, int D, int PHI>
cudaError_t launch_sweep(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const float* prefix,
                         const float* S_in, const float* z_in, int block_tokens, int nblk, void* out, float* S_out,
                         float* z_out, cudaStream_t st) {
    constexpr size_t smem = sizeof(FwdSmem<T, D>);
    static_assert(smem <= 227 * 1024, "shared memory");
    const cudaError_t e = ensure_smem<gated_sweep_kernel<T, D, PHI>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(gated_sweep_kernel<T, D, PHI>, dim3((unsigned)nblk, (unsigned)p.bh()), dim3(Shape<T, D>::THREADS),
                      smem, st, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                      gates, prefix, S_in, z_in, p.N, block_tokens, nblk, p.normalize,
                      static_cast<T*>(out), S_out, z_out);
}

template <typename T, int D, int PHI>
cudaError_t launch_states(const Problem& p, bool reverse, const void* x, const void* y, const uint8_t* gates,
                          const float* up, const float* col, int block_tokens, int nblk, int blk0, int count, bool exact, float* rec, float* dec,
                          cudaStream_t st) {
    constexpr size_t smem = sizeof(StateSmem<T, D>);
    static_assert(smem <= 227 * 1024, "shared memory");
    const dim3 grid((unsigned)count, (unsigned)p.bh());
    if (reverse) {
        const cudaError_t e = ensure_smem<gated_state_kernel<T, D, PHI, true>>(smem);
        if (e != cudaSuccess) return e;
        return launch_pdl(gated_state_kernel<T, D, PHI, true>, grid, dim3(Shape<T, D>::THREADS), smem, st,
                          static_cast<const T*>(x), static_cast<const T*>(y), gates, up, col, p.N,
                          block_tokens, nblk, blk0, exact, rec, dec);
    }
    const cudaError_t e = ensure_smem<gated_state_kernel<T, D, PHI, false>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(gated_state_kernel<T, D, PHI, false>, grid, dim3(Shape<T, D>::THREADS), smem, st,
                      static_cast<const T*>(x), static_cast<const T*>(y), gates, up, col, p.N,
                      block_tokens, nblk, blk0, exact, rec, dec);
}

}  // namespace gated

template <typename T>
cudaError_t gated_sweep_t(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const float* prefix,
                          const float* S_in, const float* z_in, int block_tokens, int nblk, void* out, float* S_out,
                          float* z_out, cudaStream_t st) {
    return gated::dispatch(p, [&](auto d, auto phi) -> cudaError_t {
        constexpr int D = decltype(d)::value;
        if constexpr (sizeof(T) == 2 && D == 128)  // tc_gated_sweep's
            return cudaErrorInvalidValue;
        else
            return gated::launch_sweep<T, D, decltype(phi)::value>(p, q, k, v, gates, prefix, S_in, z_in, block_tokens, nblk,
                                                                   out, S_out, z_out, st);
    });
}
template <typename T>
cudaError_t gated_states_t(const Problem& p, bool reverse, const void* x, const void* y, const uint8_t* gates,
                           const float* up, const float* col, int block_tokens, int nblk, int blk0, int count, bool exact, float* rec, float* dec,
                           cudaStream_t st) {
    return gated::dispatch(p, [&](auto d, auto phi) {
        return gated::launch_states<T, decltype(d)::value, decltype(phi)::value>(p, reverse, x, y, gates, up, col, block_tokens,
                                                                                nblk, blk0, count, exact, rec, dec, st);
    });
}

}  // namespace la
