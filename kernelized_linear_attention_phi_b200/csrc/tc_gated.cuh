// Pieces shared by the tcgen05 kernels of gated linear attention (bf16).
#pragma once

#include "gate_scan.cuh"
#include "launch_util.h"
#include "tc.h"
#include "tc_common.cuh"

namespace la {
namespace tcg {

using namespace tc;

// The decays of queries below 2^-60 are taken apart from the state's (tc_gated.cu).
constexpr float kDeep = -60.f;

// Brings a box of a tensor map towards L2, ahead of its load.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// Warp-wide, M = 64 accumulators: lanes 0..15 receive TMEM lane (base + i),
// columns [col, col + 8), lanes 16..31 TMEM lane (base + i - 16), columns
// [col + SPLIT, col + SPLIT + 8).
template <int SPLIT> __device__ __forceinline__ void tmem_ld8x2(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr), "n"(SPLIT));
}

// One arrival for the whole warp, behind all its lanes' accesses (each lane has
// fenced what needs a fence): barriers count warps, since an arrival per thread
// costs the shared-memory pipe a turn per thread.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// The warp's index, through a shuffle: the compiler then knows that it is the
// same in all lanes and that branches on it do not split the warp.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0); }

// One lane of a converged warp. The warp runs its loops and waits as a whole and
// only the issue is this lane's, which lets the compiler keep descriptors and
// loop counters in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^n as two bf16 in one word, n the whole part of a query's decay b that its
// features take (0 unless the chunk is steep), and n from the word.
constexpr float kSteep = -16.f;
constexpr uint32_t kOne2 = 0x3f803f80u;
__device__ __forceinline__ uint32_t whole_pow2(float b, bool steep) {
    return steep ? (uint32_t)((int)rintf(fmaxf(fminf(b, 0.f), kDeep)) + 127) * 0x00800080u : kOne2;
}
__device__ __forceinline__ float whole_bits(uint32_t word) { return (float)((int)(word >> 23) - 127); }
// Eight bf16 values times 2^n (exact while they stay in the normal range).
__device__ __forceinline__ uint4 scale8(const uint4& x, uint32_t pow2) {
    const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162*>(&pow2);
    uint4 r = x;
    uint32_t* w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(w + i), s);
        w[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    return r;
}

// The two gates of this lane (tokens row0 + 2 lane, + 1; 0 past the row's end),
// as loaded: converting them here would wait for the load.
struct Gates2 {
    uint16_t g[2];
};
__device__ __forceinline__ Gates2 load_gates(const __nv_bfloat16* g, int row0, int end, int lane) {
    const int i = row0 + 2 * lane;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(g) + i;
    Gates2 r{{0, 0}};
    if (i < end) asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(r.g[0]) : "l"(p));
    if (i + 1 < end) asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(r.g[1]) : "l"(p + 1));
    return r;
}

template <int PHI> __device__ __forceinline__ float phi_f32(float x) {
    if constexpr (PHI == PHI_RELU1) return relu_nan(x) + 1.f;
    if constexpr (PHI == PHI_ELU1) return x > 0.f ? x + 1.f : ex2(x * 1.4426950408889634f);
    return x;
}
// x + 1 of eight bf16 values, rounded to bf16.
__device__ __forceinline__ uint4 plus_one8(const uint4& x) {
    uint4 r = x;
    uint32_t* w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(w + i), __float2bfloat162_rn(1.f));
        w[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    return r;
}
// phi(x) of eight bf16 values (rounded to bf16), and w phi(x) in fp32 (f), as a
// bf16 part and the bf16 of what it leaves.
template <int PHI>
__device__ __forceinline__ void weighted8(const uint4& x, float w, float (&f)[8], uint4& phi, uint4& hi, uint4& lo) {
    if constexpr (PHI == PHI_RELU1) {  // w (relu(x) + 1) = w relu(x) + w; relu(x) is exact in bf16
        const uint4 r = make_uint4(relu_nan_x2(x.x), relu_nan_x2(x.y), relu_nan_x2(x.z), relu_nan_x2(x.w));
        phi = plus_one8(r);
        unpack8(r, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf(f[e], w, w);
    } else {
        unpack8(x, f);
        if constexpr (PHI == PHI_ELU1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = phi_f32<PHI>(f[e]);
            phi = pack8(f);
        } else {
            phi = x;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= w;
    }
    hi = pack8(f);
    float h[8];
    unpack8(hi, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = f[e] - h[e];
    lo = pack8(h);
}
// phi(x) of eight bf16 values, rounded to bf16.
template <int PHI> __device__ __forceinline__ uint4 phi_round8(const uint4& x) {
    if constexpr (PHI == PHI_ELU1) {
        float f[8];
        unpack8(x, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = phi_f32<PHI>(f[e]);
        return pack8(f);
    }
    if constexpr (PHI == PHI_RELU1)
        return plus_one8(make_uint4(relu_nan_x2(x.x), relu_nan_x2(x.y), relu_nan_x2(x.z), relu_nan_x2(x.w)));
    return x;
}

}  // namespace tcg
}  // namespace la
