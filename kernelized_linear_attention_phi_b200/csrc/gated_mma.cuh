// Warp-level matrix tiles of the gated kernels (gated_fwd.cuh, gated_bwd.cuh).
//
// One 16 x 16 x 8 step of C += A B on the warp's matrix instructions, for two
// element types with one lane layout. With g = lane / 4, t = lane % 4:
//   A (16 x 16): lane holds rows g, g + 8, columns 2t, 2t + 1, 2t + 8, 2t + 9;
//   B (16 x 8):  rows 2t, 2t + 1, 2t + 8, 2t + 9 of column g;
//   C (16 x 8):  rows g, g + 8, columns 2t, 2t + 1.
// An accumulator pair (16 columns) is therefore an A operand of the next
// product with no data moved between lanes.
//   bf16: mma.m16n8k16, fp32 accumulation.
//   fp32: mma.m16n8k8 in tf32 on two-part operands, x = hi + lo with hi the
//     nearest tf32 value, as hi*hi + hi*lo + lo*hi: the dropped lo*lo and the
//     rounding of lo are at most 2^-23 of the product and of either sign, so
//     the sums are fp32 sums. The order of k inside a step is free, so logical
//     k = 2t, 2t + 1 take the instruction's k = t, t + 4 and both types share
//     the layout.
// These are not the tensor cores' fastest instructions. Their rate alone would do
// at the intensity of this method (about 60 flop per byte: 8 cycles for
// 16 x 8 x 16 on a quarter of an SM, 1300 cycles for a chunk at d = 64), but every
// operand comes out of shared memory, and that is what the kernels wait for (68 %
// busy at 38 % of a copy's rate, 4x16x8192x64 forward). The state and the decayed
// products stay in registers between them, where the decay changes them every
// chunk. d = 128 in bf16 runs on tcgen05 going forward (tc_gated.cu).
#pragma once

#include "common.cuh"
#include "gate_scan.cuh"

namespace la {
namespace gated {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <typename T> struct FragA;
template <typename T> struct FragB;
template <> struct FragA<__nv_bfloat16> { uint32_t r[4]; };
template <> struct FragB<__nv_bfloat16> { uint32_t r[2]; };
template <> struct FragA<float> { float r[8]; };  // (g: 2t, 2t+1), (g+8: same), (g: 2t+8, 2t+9), (g+8: same)
template <> struct FragB<float> { float r[4]; };  // rows 2t, 2t+1, 2t+8, 2t+9

__device__ __forceinline__ void mma_step(float (&c)[4], const FragA<__nv_bfloat16>& a, const FragB<__nv_bfloat16>& b) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.r[0]), "r"(a.r[1]), "r"(a.r[2]), "r"(a.r[3]), "r"(b.r[0]), "r"(b.r[1]));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Nearest tf32 (the instruction drops the low 13 bits itself; half of their
// range is added before). The rest has 12 bits m at most, 2^11 <= m < 2^12, and
// the instruction keeps 11: m + m / 2^11 lies in [m + 1, m + 2), so an odd m is
// cut to m + 1 and an even one to m, which rounds it; where x is a NaN, both
// parts together keep one (an integer addition would carry out of it).
__device__ __forceinline__ uint32_t tf32_hi(float x) { return (__float_as_uint(x) + 0x1000u) & 0xffffe000u; }
__device__ __forceinline__ uint32_t tf32_lo(float x) {
    return __float_as_uint((x - __uint_as_float(tf32_hi(x))) * (1.f + 1.f / 2048));
}
// The instruction's own additions cut off what falls below the sum: the steps'
// sums are added here, rounded to nearest.
__device__ __forceinline__ void mma_step(float (&c)[4], const FragA<float>& a, const FragB<float>& b) {
    float s[4] = {};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float* x = a.r + 4 * h;
        const uint32_t h0 = tf32_hi(x[0]), h1 = tf32_hi(x[2]), h2 = tf32_hi(x[1]), h3 = tf32_hi(x[3]);
        const uint32_t y0 = tf32_hi(b.r[2 * h]), y1 = tf32_hi(b.r[2 * h + 1]);
        mma_tf32(s, tf32_lo(x[0]), tf32_lo(x[2]), tf32_lo(x[1]), tf32_lo(x[3]), y0, y1);
        mma_tf32(s, h0, h1, h2, h3, tf32_lo(b.r[2 * h]), tf32_lo(b.r[2 * h + 1]));
        mma_tf32(s, h0, h1, h2, h3, y0, y1);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] += s[e];
}

// ---- lane values of A and B operands as floats, and back -----------------------
__device__ __forceinline__ void unpack(const FragA<__nv_bfloat16>& a, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(a.r[i]);
        f[2 * i + 1] = bf16_hi(a.r[i]);
    }
}
__device__ __forceinline__ void unpack(const FragA<float>& a, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = a.r[i];
}
// The operand nearest to f (bf16: rounded once).
__device__ __forceinline__ void make_a(FragA<__nv_bfloat16>& a, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a.r[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
}
__device__ __forceinline__ void make_a(FragA<float>& a, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a.r[i] = f[i];
}
// An accumulator pair (columns 0..7 in c0, 8..15 in c1) as the next A operand.
template <typename T>
__device__ __forceinline__ void make_a(FragA<T>& a, const float (&c0)[4], const float (&c1)[4]) {
    const float f[8] = {c0[0], c0[1], c0[2], c0[3], c1[0], c1[1], c1[2], c1[3]};
    make_a(a, f);
}
// f as hi + lo bf16 operands (16 of the 24 bits of fp32: the error left is
// 2^-17 of the value); fp32 operands hold f as it is and lo is unused.
__device__ __forceinline__ void split_a(FragA<__nv_bfloat16>& hi, FragA<__nv_bfloat16>& lo, const float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi.r[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
        lo.r[i] = pack_bf16(f[2 * i] - bf16_lo(hi.r[i]), f[2 * i + 1] - bf16_hi(hi.r[i]));
    }
}
__device__ __forceinline__ void split_a(FragA<float>& hi, FragA<float>&, const float (&f)[8]) { make_a(hi, f); }
// The last 8 bits: what split_a leaves.
__device__ __forceinline__ void rest_a(FragA<__nv_bfloat16>& rest, const float (&f)[8]) {
    FragA<__nv_bfloat16> hi, lo;
    split_a(hi, lo, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        rest.r[i] = pack_bf16((f[2 * i] - bf16_lo(hi.r[i])) - bf16_lo(lo.r[i]),
                              (f[2 * i + 1] - bf16_hi(hi.r[i])) - bf16_hi(lo.r[i]));
}

// ---- feature map on operands ------------------------------------------------------
// Rounded to the operand's type: relu(x) + 1 in packed bf16 arithmetic equals
// the fp32 value rounded once.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^x of x <= 0 as 2^(x log2 e): 2^-22 of the value, and 2^-24 |x| from the product's rounding.
__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(x * 1.4426950408889634f); }
template <int PHI> __device__ __forceinline__ float phi_f(float x) {
    if (PHI == PHI_RELU1) return relu_nan(x) + 1.f;
    if (PHI == PHI_ELU1) return x > 0.f ? x + 1.f : exp_fast(x);
    return x;
}
// d phi / dx, at 0 as in phi_grad (common.cuh)
template <int PHI> __device__ __forceinline__ float slope_f(float x) {
    if (PHI == PHI_RELU1) return x > 0.f ? 1.f : 0.f;
    if (PHI == PHI_ELU1) return x > 0.f ? 1.f : exp_fast(x);
    return 1.f;
}
template <int PHI> __device__ __forceinline__ uint32_t phi_pair(uint32_t w) {
    if (PHI == PHI_RELU1) {
        w = relu_nan_x2(w);
        const __nv_bfloat162 x = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(1.f));
        return *reinterpret_cast<const uint32_t*>(&x);
    }
    if (PHI == PHI_ELU1) return pack_bf16(phi_f<PHI>(bf16_lo(w)), phi_f<PHI>(bf16_hi(w)));
    return w;
}
// phi(x) - shift with shift = 1 for the maps that end in + 1, else 0: relu(x),
// which bf16 holds exactly, elu(x), or x. A product with phi(x) is the product
// with base(x) plus the sum over k of the other factor, taken in fp32: the
// rounding of the other factor then multiplies only base(x), not the part
// that all rows share, which the gradients of q cancel.
template <int PHI> constexpr bool shifted = PHI != PHI_IDENTITY;
template <int PHI> __device__ __forceinline__ float base_f(float x) {
    if (PHI == PHI_RELU1) return relu_nan(x);
    if (PHI == PHI_ELU1) return x > 0.f ? x : exp_fast(x) - 1.f;
    return x;
}
template <int PHI> __device__ __forceinline__ uint32_t base_pair(uint32_t w) {
    if (PHI == PHI_RELU1) return relu_nan_x2(w);
    if (PHI == PHI_ELU1) return pack_bf16(base_f<PHI>(bf16_lo(w)), base_f<PHI>(bf16_hi(w)));
    return w;
}
template <int PHI> __device__ __forceinline__ void base_frag(FragB<__nv_bfloat16>& b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) b.r[i] = base_pair<PHI>(b.r[i]);
}
template <int PHI> __device__ __forceinline__ void base_frag(FragB<float>& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b.r[i] = base_f<PHI>(b.r[i]);
}
template <int PHI> __device__ __forceinline__ void phi_frag(FragA<__nv_bfloat16>& a) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a.r[i] = phi_pair<PHI>(a.r[i]);
}
template <int PHI> __device__ __forceinline__ void phi_frag(FragB<__nv_bfloat16>& b) {
#pragma unroll
    for (int i = 0; i < 2; ++i) b.r[i] = phi_pair<PHI>(b.r[i]);
}
template <int PHI> __device__ __forceinline__ void phi_frag(FragA<float>& a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) a.r[i] = phi_f<PHI>(a.r[i]);
}
template <int PHI> __device__ __forceinline__ void phi_frag(FragB<float>& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b.r[i] = phi_f<PHI>(b.r[i]);
}

// ---- phi(x) . phi(y) without phi's rounding, for the gradients ---------------------------
// What all channels share cancels in the gradients, and 1 + x rounded to bf16 has
// lost most of a small x by then (sigma 0.02, 2 x 4 x 500 x 64, relu + 1: dq 1.6e-2
// off with phi as the operand, 1.7e-3 as here). relu + 1: phi = 1 + base with base
// exact in bf16, sum (1 + b_x)(1 + b_y) = D + sum b_x + sum b_y + sum b_x b_y, the
// ones as an operand. elu + 1 (whose 1 + base would lose the small phi of far
// negative x): phi in two bf16 parts. fp32 holds phi as it is.
template <int D, int PHI> struct PhiDot {
    // the rows' part, ones(phi(x)): added up by `rows` from every raw A operand of x; phi(x) . z with z a
    // load_column and sz the sum of z
    template <typename T> __device__ __forceinline__ static void rows(float (&s)[4], const FragA<T>& x) {
        if constexpr (sizeof(T) == 2 && PHI == PHI_RELU1) {
            FragA<T> a = x;
            const FragB<T> ones{{0x3f803f80u, 0x3f803f80u}};
#pragma unroll
            for (int i = 0; i < 4; ++i) a.r[i] = base_pair<PHI>(a.r[i]);
            mma_step(s, a, ones);
        }
    }
    // p before the products: two accumulators of 8 columns
    template <typename T> __device__ __forceinline__ static void start(float (&p)[2][4], const float (&s)[4]) {
        constexpr bool APART = sizeof(T) == 2 && PHI == PHI_RELU1;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            p[n][0] = p[n][1] = APART ? s[0] + D : 0.f;
            p[n][2] = p[n][3] = APART ? s[2] + D : 0.f;
        }
    }
    // p += the products of one step's raw operands
    __device__ __forceinline__ static void step(float (&p)[2][4], FragA<float> a, FragB<float> (&b)[2]) {
        phi_frag<PHI>(a);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            phi_frag<PHI>(b[n]);
            mma_step(p[n], a, b[n]);
        }
    }
    __device__ __forceinline__ static void step(float (&p)[2][4], FragA<__nv_bfloat16> a, FragB<__nv_bfloat16> (&b)[2]) {
        if constexpr (PHI == PHI_ELU1) {
            FragA<__nv_bfloat16> lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) split_phi(a.r[i], a.r[i], lo.r[i]);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                FragB<__nv_bfloat16> bl;
#pragma unroll
                for (int i = 0; i < 2; ++i) split_phi(b[n].r[i], b[n].r[i], bl.r[i]);
                mma_step(p[n], lo, b[n]);
                mma_step(p[n], a, bl);
                mma_step(p[n], a, b[n]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) a.r[i] = base_pair<PHI>(a.r[i]);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                base_frag<PHI>(b[n]);
                if constexpr (PHI == PHI_RELU1) {
                    const FragA<__nv_bfloat16> ones{{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}};
                    mma_step(p[n], ones, b[n]);
                }
                mma_step(p[n], a, b[n]);
            }
        }
    }
    // s += phi(x) z (relu + 1: without the ones' part, the sum of z)
    __device__ __forceinline__ static void column(float (&s)[4], FragA<float> x, const FragB<float>& z) {
        phi_frag<PHI>(x);
        mma_step(s, x, z);
    }
    __device__ __forceinline__ static void column(float (&s)[4], FragA<__nv_bfloat16> x, const FragB<__nv_bfloat16>& z) {
        if constexpr (PHI == PHI_ELU1) {
            FragA<__nv_bfloat16> lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) split_phi(x.r[i], x.r[i], lo.r[i]);
            mma_step(s, lo, z);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x.r[i] = base_pair<PHI>(x.r[i]);
        }
        mma_step(s, x, z);
    }
    __device__ __forceinline__ static void split_phi(uint32_t w, uint32_t& hi, uint32_t& lo) {
        const float x = phi_f<PHI>(bf16_lo(w)), y = phi_f<PHI>(bf16_hi(w));
        hi = pack_bf16(x, y);
        lo = pack_bf16(x - bf16_lo(hi), y - bf16_hi(hi));
    }
};

// ---- operands from shared-memory tiles [rows][LD] --------------------------------------
// LD is 16 bytes (bf16) or 32 bytes (fp32) more than the row, so the 8 rows an
// access touches start in different banks (the scalar fp32 loads down a
// column meet two lanes to a bank).
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)) : "memory");
}

// A = tile[m0 .. m0 + 15][k0 .. k0 + 15]
template <int LD>
__device__ __forceinline__ void load_a(FragA<__nv_bfloat16>& a, const __nv_bfloat16* tile, int m0, int k0, int lane) {
    ldsm4(a.r, tile + (m0 + (lane & 7) + ((lane >> 3) & 1) * 8) * LD + k0 + (lane >> 4) * 8);
}
template <int LD>
__device__ __forceinline__ void load_a(FragA<float>& a, const float* tile, int m0, int k0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 x = *reinterpret_cast<const float2*>(tile + (m0 + g) * LD + k0 + 8 * h + 2 * t);
        const float2 y = *reinterpret_cast<const float2*>(tile + (m0 + g + 8) * LD + k0 + 8 * h + 2 * t);
        a.r[4 * h] = x.x; a.r[4 * h + 1] = x.y; a.r[4 * h + 2] = y.x; a.r[4 * h + 3] = y.y;
    }
}
// A = transpose of tile[k0 .. k0 + 15][m0 .. m0 + 15]
template <int LD>
__device__ __forceinline__ void load_at(FragA<__nv_bfloat16>& a, const __nv_bfloat16* tile, int k0, int m0, int lane) {
    ldsm4_t(a.r, tile + (k0 + (lane & 7) + (lane >> 4) * 8) * LD + m0 + ((lane >> 3) & 1) * 8);
}
template <int LD>
__device__ __forceinline__ void load_at(FragA<float>& a, const float* tile, int k0, int m0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float* row = tile + (k0 + 8 * h + 2 * t + j) * LD + m0 + g;
            a.r[4 * h + j] = row[0];
            a.r[4 * h + 2 + j] = row[8];
        }
}
// Two B operands (columns n0 .. n0 + 7 and n0 + 8 .. n0 + 15) of the transpose
// of tile[n0 .. n0 + 15][k0 .. k0 + 15]
template <int LD>
__device__ __forceinline__ void load_bt(FragB<__nv_bfloat16> (&b)[2], const __nv_bfloat16* tile, int n0, int k0, int lane) {
    uint32_t r[4];
    ldsm4(r, tile + (n0 + (lane & 7) + (lane >> 4) * 8) * LD + k0 + ((lane >> 3) & 1) * 8);
    b[0].r[0] = r[0]; b[0].r[1] = r[1]; b[1].r[0] = r[2]; b[1].r[1] = r[3];
}
template <int LD>
__device__ __forceinline__ void load_bt(FragB<float> (&b)[2], const float* tile, int n0, int k0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 x = *reinterpret_cast<const float2*>(tile + (n0 + 8 * p + g) * LD + k0 + 8 * h + 2 * t);
            b[p].r[2 * h] = x.x;
            b[p].r[2 * h + 1] = x.y;
        }
}
// Two B operands of tile[k0 .. k0 + 15][n0 .. n0 + 15]
template <int LD>
__device__ __forceinline__ void load_b(FragB<__nv_bfloat16> (&b)[2], const __nv_bfloat16* tile, int k0, int n0, int lane) {
    uint32_t r[4];
    ldsm4_t(r, tile + (k0 + (lane & 7) + ((lane >> 3) & 1) * 8) * LD + n0 + (lane >> 4) * 8);
    b[0].r[0] = r[0]; b[0].r[1] = r[1]; b[1].r[0] = r[2]; b[1].r[1] = r[3];
}
template <int LD>
__device__ __forceinline__ void load_b(FragB<float> (&b)[2], const float* tile, int k0, int n0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float* row = tile + (k0 + 8 * h + 2 * t + j) * LD + n0 + g;
            b[0].r[2 * h + j] = row[0];
            b[1].r[2 * h + j] = row[8];
        }
}
// A B operand whose column 0 is x[k0 .. k0 + 15] (fp32, shared memory) and
// whose column 1 is what bf16 rounding left of it; the other columns are 0.
__device__ __forceinline__ void load_column(FragB<__nv_bfloat16>& b, const float* x, int k0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 f = *reinterpret_cast<const float2*>(x + k0 + 8 * h + 2 * t);
        const uint32_t hi = pack_bf16(f.x, f.y);
        const uint32_t lo = pack_bf16(f.x - bf16_lo(hi), f.y - bf16_hi(hi));
        b.r[h] = g == 0 ? hi : g == 1 ? lo : 0u;
    }
}
__device__ __forceinline__ void load_column(FragB<float>& b, const float* x, int k0, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 f = *reinterpret_cast<const float2*>(x + k0 + 8 * h + 2 * t);
        b.r[2 * h] = g == 0 ? f.x : 0.f;
        b.r[2 * h + 1] = g == 0 ? f.y : 0.f;
    }
}

// ---- asynchronous copies ------------------------------------------------------------------
// 16 bytes, or 16 zero bytes when !in (then `src` is not read).
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float quad_sum(float x) {  // over the 4 lanes that share a row
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

}  // namespace gated
}  // namespace la
