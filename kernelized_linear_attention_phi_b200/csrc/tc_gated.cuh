// Pieces shared by the tcgen05 kernels of gated linear attention (bf16).
#pragma once

#include "launch_util.h"
#include "tc.h"
#include "tc_common.cuh"

namespace la {
namespace tcg {

using namespace tc;

// Log-gates of a chunk of 64 tokens, in units of log2. A closed gate (-inf)
// counts as 2^-160, which fp32 cannot hold: every product across it is 0. The
// sums are formed in 64 bits; kept as fp32 they blur a decay by 2^-24 of the
// chunk's whole sum, below the rounding of bf16 results even with some ten
// closed gates in one chunk.
constexpr float kClosedLog2 = -160.f;
// Queries whose products reach below 2^-90 are scaled by 2^90 (tc_gated.cu).
constexpr float kDeep = -90.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The two gates of this lane (tokens row0 + 2 lane, + 1), 0 past the row's end.
__device__ __forceinline__ float2 load_gates(const __nv_bfloat16* g, int row0, int end, int lane) {
    const int i = row0 + 2 * lane;
    return make_float2(i < end ? __bfloat162float(g[i]) : 0.f, i + 1 < end ? __bfloat162float(g[i + 1]) : 0.f);
}
// A whole warp: inclusive sums (log2) of this lane's two tokens over the chunk.
// Returns the chunk's sum.
__device__ __forceinline__ double scan_gates(float2 g, int lane, double& b0, double& b1) {
    constexpr double kLog2e = 1.4426950408889634;
    double x = (double)g.x * kLog2e, y = (double)g.y * kLog2e;
    x = x < kClosedLog2 ? kClosedLog2 : x;  // a NaN stays
    y = y < kClosedLog2 ? kClosedLog2 : y;
    double run = x + y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
    }
    b1 = run;
    b0 = run - y;
    return __shfl_sync(0xffffffffu, run, 31);
}

template <int PHI> __device__ __forceinline__ float phi_f32(float x) {
    if constexpr (PHI == PHI_RELU1) return fmaxf(x, 0.f) + 1.f;
    if constexpr (PHI == PHI_ELU1) return x > 0.f ? x + 1.f : ex2(x * 1.4426950408889634f);
    return x;
}
// w phi(x) of eight bf16 values in fp32 (f), as a bf16 part and the bf16 of what it leaves.
template <int PHI>
__device__ __forceinline__ void weighted8(const uint4& x, float w, float (&f)[8], uint4& hi, uint4& lo) {
    unpack8(x, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = phi_f32<PHI>(f[e]) * w;
    hi = pack8(f);
    float h[8];
    unpack8(hi, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = f[e] - h[e];
    lo = pack8(h);
}

}  // namespace tcg
}  // namespace la
