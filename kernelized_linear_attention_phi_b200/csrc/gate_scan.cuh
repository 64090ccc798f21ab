// Running sums of the log-gates of a chunk by one warp, in units of log2 and
// fixed point (31 bits behind the point). Integer sums are exact: the decay
// between two tokens depends on the gates between them and on nothing else,
// however far the chunk has decayed before, and a closed gate drops out of every
// difference behind it. A gate itself is rounded to the nearest: 2^-32, or 2^-25
// of its fraction where that is more.
#pragma once

#include "common.cuh"

namespace la {

// relu(x) with a NaN left as it is, as in the other feature maps (max.f32 would
// drop it, and a head would go on as if the token's features were ones).
__device__ __forceinline__ float relu_nan(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t relu_nan_x2(uint32_t w) {  // two bf16
    const __nv_bfloat162 x = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(0.f));
    return *reinterpret_cast<const uint32_t*>(&x);
}

// Gates below this many bits count as closed: fp32 cannot hold any product
// across one (and 64 of them stay far inside the integer part).
constexpr float kClosedBits = -14000.f;

__device__ __forceinline__ long long gate_bits(float g) {
    constexpr float kHi = 1.44269504f, kLo = 1.92596299e-8f;  // log2 e in two parts
    float x = g * kHi;
    const float rest = fmaf(g, kHi, -x) + g * kLo;
    if (!(x >= kClosedBits)) return (long long)(int)kClosedBits << 31;  // -inf too (a NaN is dealt with by the caller)
    const float n = rintf(fminf(x, 16000.f));
    const float f = (fminf(x, 16000.f) - n) + rest;  // at most half, and a little
    return ((long long)(int)n << 31) + __float2int_rn(f * 2147483648.f);
}
// The sum with a further chunk's b. It stops at 2^20 bits either way, where
// fp32 has long reached 0 or infinity: without an end 150,000 closed gates
// leave the 32 bits in front of the point, and twice as many the 64 in all.
__device__ __forceinline__ long long gate_add(long long sum, long long b) {
    constexpr long long kMost = 1LL << 51;
    sum += b;
    return sum < -kMost ? -kMost : sum > kMost ? kMost : sum;
}
// 2^b: the fraction alone goes through the fp32 function.
__device__ __forceinline__ float gate_pow2(long long b) {
    const long long whole = b >> 31;
    const int n = whole < -127 ? -127 : whole > 128 ? 128 : (int)whole;
    const float f = (float)((int)b & 0x7fffffff) * 4.65661287e-10f;  // 2^-31
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(f));
    return n < -126 ? 0.f : n > 127 ? INFINITY : y * __int_as_float((n + 127) << 23);
}
// b as hi + lo
__device__ __forceinline__ float2 gate_float2(long long b) {
    const float n = (float)(int)(b >> 31), f = (float)((int)b & 0x7fffffff) * 4.65661287e-10f;
    const float hi = n + f;
    return make_float2(hi, (n - hi) + f);
}

__device__ __forceinline__ float gate_value(uint32_t fp32) { return __uint_as_float(fp32); }
__device__ __forceinline__ float gate_value(uint16_t bf16) { return __uint_as_float((uint32_t)bf16 << 16); }

// A whole warp: the sums of a lane's R consecutive tokens (inclusive) and of
// the chunk of 32 R, from the gates as they were loaded. `bad`: bit e, a NaN or
// +inf among the gates up to token e; bit R, one in the chunk.
template <int R> struct GateSums {
    long long b[R], last;
    int bad;
};
template <int R, typename Raw>
__device__ __forceinline__ GateSums<R> sum_gates(const Raw (&g)[R], int lane) {
    GateSums<R> s;
    long long run = 0;
    int bad = 0;
#pragma unroll
    for (int e = 0; e < R; ++e) {
        const float x = gate_value(g[e]);
        bad |= (x < INFINITY ? 0 : 1) << e;
        run += gate_bits(x);
        s.b[e] = run;
    }
    const long long own = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
    }
    s.last = __shfl_sync(0xffffffffu, run, 31);
    const unsigned any = __ballot_sync(0xffffffffu, bad != 0);
    s.bad = any ? 1 << R : 0;
    bool upto = any & ((1u << lane) - 1u);
#pragma unroll
    for (int e = 0; e < R; ++e) {
        s.b[e] += run - own;
        upto = upto || bad & (1 << e);
        s.bad |= (upto ? 1 : 0) << e;
    }
    return s;
}

}  // namespace la
