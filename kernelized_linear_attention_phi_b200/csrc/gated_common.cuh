// What the gated kernels share: tile shapes, the gates of a chunk as sums of
// logarithms, tile loads, and the state's update.
#pragma once

#include <cstddef>

#include "gated_mma.cuh"
#include "internal.h"

namespace la {
namespace gated {

// Tile shapes per element type and d. A chunk has C tokens; NW warps split
// it into RG row groups of 16 tokens and CG column groups of NCOL channels.
// The state S (d x d, fp32) lives in the warps' registers: SRT row tiles of
// 16, each cut into SCG column groups of SN columns. SB: operand copies of S
// in shared memory, ST: chunks of tiles. What bounds these kernels is the
// latency of one warp's chain of loads, products and barriers (4x16x8192x64
// bf16, forward: the tensor pipe busy a quarter of the time, issue slots a
// third). At d <= 64 one S and one chunk leave room for three or four CTAs
// per SM, which cover for each other (with two chunks and two or three CTAs the
// forward sweep takes 121 us, so 109; dk and dv 254, so 223); twice the warps on
// a chunk gain nothing, since each then repeats more (194 us). At d = 128 an
// SM holds one CTA, which loads a chunk ahead. fp32 rows are twice as long, so
// d >= 64 takes chunks of 32 tokens.
template <typename T, int D> struct Shape {
    static constexpr bool F32 = sizeof(T) == 4;
    static constexpr int C = F32 && D >= 64 ? 32 : 64;
    static constexpr int NW = D == 128 ? 8 : 4;
    static constexpr int SB = F32 || D <= 64 ? 1 : 2;
    static constexpr int ST = D == 128 ? 2 : 1;
    static constexpr int THREADS = NW * 32;
    static constexpr int LD = D + 8;
    static constexpr int EPV = 16 / sizeof(T);
    static constexpr int RG = C / 16, CG = NW / RG, NCOL = D / CG;
    static constexpr int SRT = D / 16 < NW ? D / 16 : NW;
    static constexpr int SCG = (NW / SRT) < (D / 16) ? (NW / SRT) : (D / 16);
    static constexpr int SN = D / SCG;
    static constexpr int TILE = C * LD;  // elements of a [C x D] tile
    static constexpr int SOP = D * LD;   // elements of the S operand
    static_assert(RG * CG == NW && SRT * 16 == D && NCOL % 16 == 0, "tiles");
};

// The row group of a warp. Row groups see one to RG key groups, so the order is
// turned from CTA to CTA, and reversed for a CTA's second four warps: an SM's
// four schedulers get the same work (gradient sweeps of 1x16x32768x128 bf16: 422
// us -> 390 and 537 -> 498; 1x16x8192x128 fp32 forward 381 -> 356).
template <typename SH> __device__ __forceinline__ int row_group(int warp) {
    const int x = (warp + blockIdx.x + blockIdx.y) % SH::RG;
    return warp & 4 ? SH::RG - 1 - x : x;
}

// The gates of one chunk, from b_i = log2 of the product of the chunk's gates
// up to token i (gate_scan.cuh). The decay from key j to query i, 2^(b_i - b_j),
// is the product of from_start_i and inv_j while every b of the chunk lies
// within 90 of 0 (deep = 0). In a deep chunk it is formed per pair from
// b = hi + lo. The two factors meet before either touches a product of tokens:
// inv_j is up to 2^90, and (phi(q_i).phi(k_j)) inv_j v_j would leave fp32 for
// products of some 2^37, as 2^-90 of a small upstream gradient would leave its
// normal range.
// They are computed once per call for all chunks (gates_kernel, gated.cu) and
// come with the tiles: forming them inside a sweep puts a warp's scan on
// every chunk's way.
template <int C> struct alignas(16) Gates {
    float hi[C], lo[C];
    float from_start[C];  // 2^b_i; 0 past the last token
    float inv[C];         // 2^-b_j
    float to_end[C];      // 2^(b_last - b_j); 0 past the last token
    float all;            // 2^b_last
    int deep, pad[2];
    // second sweep, normalized: 1 / den_i, -(out_i . dout_i) and (dout_i.v_i + col_i) / den_i; 0 past the last token
    float up[C], col[C], own[C];
};
template <int C> constexpr int kGateBytes = (5 * C + 4) * 4;  // of a chunk's record in global memory
constexpr float kDeep = 90.f;
// Starts the copy of a chunk's gates; with up (a normalized call: up, col and,
// where the second sweep takes it, own of the head, from row0 on) those too.
__device__ __forceinline__ void cp_async4(void* dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
}
template <int C>
__device__ __forceinline__ void load_gates(Gates<C>& s, const uint8_t* rec, const float* up, const float* col, const float* own, int row0, int N) {
    static_assert(offsetof(Gates<C>, up) == kGateBytes<C>, "record");
    const int u = threadIdx.x;
    if (u < kGateBytes<C> / 16) cp_async16(reinterpret_cast<uint8_t*>(&s) + u * 16, rec + u * 16, true);
    if (up && u < C) {
        const bool in = row0 + u < N;
        const int i = in ? row0 + u : 0;
        cp_async4(s.up + u, up + i, in);
        cp_async4(s.col + u, col + i, in);
        if (own) cp_async4(s.own + u, own + i, in);
    }
}

// The decay between two tokens of a deep chunk, from what (hi, lo) of the one
// and token j are apart.
template <int C> __device__ __forceinline__ float decay(const Gates<C>& s, float hi_i, float lo_i, int j) {
    return exp2_fast((hi_i - s.hi[j]) + (lo_i - s.lo[j]));
}

// Starts the copy of rows row0 .. row0 + C - 1 of a [N, D] matrix (zeros past N).
template <typename SH, typename T, int D>
__device__ __forceinline__ void load_tile(T* dst, const T* src, int row0, int N) {
    constexpr int VPR = D / SH::EPV;
#pragma unroll
    for (int u = threadIdx.x; u < SH::C * VPR; u += SH::THREADS) {
        const int row = u / VPR, col = (u % VPR) * SH::EPV;
        const bool in = row0 + row < N;
        cp_async16(dst + row * SH::LD + col, src + (size_t)(in ? row0 + row : 0) * D + col, in);
    }
}

// The state in registers: this warp's row tile and columns of S, and z in the
// lanes of column 0 (its bf16 remainder products in column 1) of one more
// accumulator. Warps past SRT * SCG hold nothing.
template <typename T, int D> struct State {
    using SH = Shape<T, D>;
    float S[SH::SN / 8][4];
    float z[4];

    __device__ __forceinline__ static int row(int warp) { return (warp % SH::SRT) * 16; }
    __device__ __forceinline__ static int col(int warp) { return (warp / SH::SRT) * SH::SN; }
    __device__ __forceinline__ static bool owns(int warp) { return warp < SH::SRT * SH::SCG; }

    // from a record (S d*d, then z d at zrec), or zero
    __device__ __forceinline__ void seed(const float* rec, const float* zrec, int warp, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < SH::SN / 8; ++n) {
            float2 x = make_float2(0.f, 0.f), y = x;
            if (rec && owns(warp)) {
                const float* p = rec + (row(warp) + g) * D + col(warp) + 8 * n + 2 * t;
                x = *reinterpret_cast<const float2*>(p);
                y = *reinterpret_cast<const float2*>(p + 8 * D);
            }
            S[n][0] = x.x; S[n][1] = x.y; S[n][2] = y.x; S[n][3] = y.y;
        }
        const bool zt = rec && owns(warp) && t == 0;
        z[0] = zt ? zrec[row(warp) + g] : 0.f;
        z[2] = zt ? zrec[row(warp) + g + 8] : 0.f;
        z[1] = z[3] = 0.f;
    }
    __device__ __forceinline__ void store(float* rec, float* zrec, int warp, int lane) const {
        if (!owns(warp)) return;
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < SH::SN / 8; ++n) {
            float* p = rec + (row(warp) + g) * D + col(warp) + 8 * n + 2 * t;
            *reinterpret_cast<float2*>(p) = make_float2(S[n][0], S[n][1]);
            *reinterpret_cast<float2*>(p + 8 * D) = make_float2(S[n][2], S[n][3]);
        }
        if (col(warp) == 0 && t == 0) {
            zrec[row(warp) + g] = z[0] + z[1];
            zrec[row(warp) + g + 8] = z[2] + z[3];
        }
    }
    // the operand of the next chunk's products: S in the element type (bf16:
    // rounded once, like every other operand of the output's products; the
    // state itself stays fp32) and, where lo is given, what that rounding
    // left; z in fp32
    template <bool LO = false>
    __device__ __forceinline__ void publish(T* sop, float* zs, int warp, int lane, T* lo = nullptr) const {
        if (!owns(warp)) return;
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int n = 0; n < SH::SN / 8; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = (row(warp) + g + 8 * h) * SH::LD + col(warp) + 8 * n + 2 * t;
                const float x = S[n][2 * h], y = S[n][2 * h + 1];
                if constexpr (SH::F32) {
                    *reinterpret_cast<float2*>(sop + at) = make_float2(x, y);
                } else {
                    const uint32_t hi = pack_bf16(x, y);
                    *reinterpret_cast<uint32_t*>(sop + at) = hi;
                    if constexpr (LO)
                        *reinterpret_cast<uint32_t*>(lo + at) = pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi));
                }
            }
        if (col(warp) == 0 && t == 0) {
            zs[row(warp) + g] = z[0] + z[1];
            zs[row(warp) + g + 8] = z[2] + z[3];
        }
    }
    // S = all S + sum_j w_j u_j phi(x_j) (x) y_j,  z = all z + sum_j w_j u_j phi(x_j) c_j
    // with x, y [C x D] tiles and w, u, c (u or c null: ones) of the chunk; z only with `with_z`. w u phi(x)
    // is formed in fp32 and multiplied as hi + lo operands, so a state of bf16
    // rows errs by 2^-17 of its terms, not by bf16's 2^-8.
    template <int PHI>
    __device__ __forceinline__ static void weighted(float (&f)[8], const T* x, const float* w, const float* u, int k0, int warp,
                                                    int lane) {
        const int t = lane & 3;
        FragA<T> a;
        load_at<SH::LD>(a, x, k0, row(warp), lane);
        unpack(a, f);
        float2 w0 = *reinterpret_cast<const float2*>(w + k0 + 2 * t);
        float2 w1 = *reinterpret_cast<const float2*>(w + k0 + 8 + 2 * t);
        if (u) {
            w0.x *= u[k0 + 2 * t]; w0.y *= u[k0 + 2 * t + 1];
            w1.x *= u[k0 + 8 + 2 * t]; w1.y *= u[k0 + 8 + 2 * t + 1];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            f[2 * r] = phi_f<PHI>(f[2 * r]) * w0.x;
            f[2 * r + 1] = phi_f<PHI>(f[2 * r + 1]) * w0.y;
            f[4 + 2 * r] = phi_f<PHI>(f[4 + 2 * r]) * w1.x;
            f[5 + 2 * r] = phi_f<PHI>(f[5 + 2 * r]) * w1.y;
        }
    }
    template <int PHI>
    __device__ __forceinline__ void update(const T* x, const T* y, const float* w, const float* u, const float* c, bool with_z,
                                           float all, int warp, int lane, bool exact = false) {
        if (!owns(warp)) return;
        constexpr int K = SH::C / 16;
        FragA<T> hi[K], lo[K];
#pragma unroll
        for (int kt = 0; kt < K; ++kt) {
            float f[8];
            weighted<PHI>(f, x, w, u, kt * 16, warp, lane);
            split_a(hi[kt], lo[kt], f);
        }
        // A chunk's sum is formed from zero and then added: the matrix
        // instructions' additions do not round to nearest, which over a
        // long row would pull every entry the same way.
#pragma unroll
        for (int n = 0; n < SH::SN / 16; ++n) {
            float s[2][4] = {};
#pragma unroll
            for (int kt = 0; kt < K; ++kt) {
                FragB<T> b[2];
                load_b<SH::LD>(b, y, kt * 16, col(warp) + 16 * n, lane);
                if constexpr (!SH::F32) {
                    mma_step(s[0], lo[kt], b[0]);
                    mma_step(s[1], lo[kt], b[1]);
                }
                mma_step(s[0], hi[kt], b[0]);
                mma_step(s[1], hi[kt], b[1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S[2 * n][e] = fmaf(S[2 * n][e], all, s[0][e]);
                S[2 * n + 1][e] = fmaf(S[2 * n + 1][e], all, s[1][e]);
            }
        }
        if (with_z && col(warp) == 0) {
            float s[4] = {};
#pragma unroll
            for (int kt = 0; kt < K; ++kt) {
                FragB<T> b;
                if (c) {
                    load_column(b, c, kt * 16, lane);
                } else {
                    const bool one = lane < 4;  // column 0 of ones
                    if constexpr (SH::F32) {
                        b.r[0] = b.r[1] = b.r[2] = b.r[3] = one ? 1.f : 0.f;
                    } else {
                        b.r[0] = b.r[1] = one ? 0x3f803f80u : 0u;
                    }
                }
                if constexpr (!SH::F32) mma_step(s, lo[kt], b);
                mma_step(s, hi[kt], b);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = fmaf(z[e], all, s[e]);
        }
        if constexpr (!SH::F32 && D != 128) {  // d = 128 bf16: a caller's state comes from tc_gated_states
            if (!exact) return;
            // a state that a caller gets: the last bits of w phi(x) too
#pragma unroll 1
            for (int kt = 0; kt < K; ++kt) {
                float f[8];
                FragA<T> rest;
                weighted<PHI>(f, x, w, u, kt * 16, warp, lane);
                rest_a(rest, f);
#pragma unroll
                for (int n = 0; n < SH::SN / 16; ++n) {
                    FragB<T> b[2];
                    load_b<SH::LD>(b, y, kt * 16, col(warp) + 16 * n, lane);
                    mma_step(S[2 * n], rest, b[0]);
                    mma_step(S[2 * n + 1], rest, b[1]);
                }
                if (with_z && col(warp) == 0) {
                    FragB<T> b;
                    b.r[0] = b.r[1] = lane < 4 ? 0x3f803f80u : 0u;
                    mma_step(z, rest, b);
                }
            }
        }
    }
};

}  // namespace gated
}  // namespace la
