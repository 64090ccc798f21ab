// Gradients of gated linear attention. With S_i, z_i the state query i reads,
// up_i = 1 / den_i, delta_i = out_i . dout_i, col_i = -delta_i (unnormalized:
// up = 1, col = 0) and G_j, h_j = sum_{i >= j} e^{b_i - b_j} up_i phi(q_i) [dout_i, col_i]:
//   dq_i = phi'(q_i) * up_i (S_i dout_i + col_i z_i)
//   dk_j = phi'(k_j) * (G_j v_j + h_j),   dv_j = G_j^T phi(k_j)
//   dg_t = a_t (<S_{t-1}, G_t> + <z_{t-1}, h_t>)
// dg over a chunk, from the state S in front of it and G behind it, with
// W_ij = e^{b_i - b_j} (phi(q_i).phi(k_j)) up_i (dout_i.v_j + col_i):
//   dg_t = sum_{i >= t} (sum_j W_ij) - sum_{j >= t} (sum_i W_ij)     pairs inside the chunk
//        + sum_{i >= t} e^{b_i} up_i phi(q_i) (S dout_i + col_i z)   queries with earlier keys
//        + sum_{j < t} e^{b_last - b_j} phi(k_j) (G v_j + h)         keys with later queries
//        + e^{b_last} (<S, G> + <z, h>)                              keys and queries outside
// No term sums over more than a chunk, so dg keeps its accuracy at any length
// (the difference of the running sums of q dq and k dk would lose it), and
// W is formed in fp32 from unrounded products.
//
// Two sweeps: chunks in order for dq (S in registers; the state in front of
// each chunk is written out for the last term, and the sums over j and the
// queries' part go to dgp), then chunks in reverse for dk, dv, dg (G in
// registers). delta_i comes out of the same pass over the keys as dq, since
//   dq_i = phi'(q_i) up_i [ X_i + e^{b_i} S dout_i - delta_i (Y_i + e^{b_i} z) ],
//   X_i = sum_j e^{b_i - b_j} (dout_i.v_j) phi(k_j),  Y_i = sum_j e^{b_i - b_j} phi(k_j).
// A query's own key (j = i) is left out of these sums and of dg's and added in
// fp32 as up_i (dout_i.v_i - delta_i) phi(k_i): under fast gates its weight is all
// but 1, the difference is formed from the sums of the other keys, and what
// would have to cancel in dg (W_ii, in the sum over i and in the one over j)
// is in neither. A normalized output makes the row sum of W 0, so that the others'
// is -W_ii.
#pragma once

#include "gated.h"
#include "gated_common.cuh"
#include "launch_util.h"

namespace la {
namespace gated {

// PARTS: operands of the state (2: rounded and remainder); COPIES of them.
template <typename T, int D, int PARTS, int COPIES> struct BwdSmem {
    using SH = Shape<T, D>;
    T tiles[SH::ST][4][SH::TILE];  // q, k, v, dout
    T sop[COPIES][PARTS][SH::SOP];
    float zs[COPIES][D];
    Gates<SH::C> gates[2];
    float row[2][SH::CG][SH::C];     // per token sums for dg
    float sum[2][SH::C];             // the keys' sums of W over the queries behind
    float part[SH::CG][SH::C];
    float dot[2][SH::NW];
};

// The first sweep subtracts delta_i z from S dout_i; with features that are
// positive (relu + 1, elu + 1) both are dominated by the part that all
// channels share, and what is left would carry the rounding of the whole: S
// goes in as two bf16 parts there (relative error of dq at 2 x 8 x 4096 x 64,
// relu + 1: 6.1e-3 with one part). Under the identity map dg needs them: the sums
// over a chunk's queries of phi(q) . (S dout) all carry the same rounding of S
// (1 x 16 x 32768 x 128: dg 2.2e-3 off with one part here and one in the records
// below, 1.7e-3 with two and fp32; 4 x 16 x 8192 x 128: sweeps 440 -> 537 and 549 -> 592 us).
template <typename T, int D, int PHI> struct BwdQ {
    static constexpr int PARTS = sizeof(T) == 2 ? 2 : 1;
    static constexpr int COPIES = D == 128 && PARTS == 2 ? 1 : Shape<T, D>::SB;
    using Smem = BwdSmem<T, D, PARTS, COPIES>;
};
template <typename T, int D> using BwdKvSmem = BwdSmem<T, D, 1, Shape<T, D>::SB>;

// State records between the sweeps, in fp32: per chunk, the fragments of S in
// thread order (both sweeps hold S and G in the same lanes), then z. dg takes
// <S, G> from them.
template <typename T, int D> struct ChunkState {
    using SH = Shape<T, D>;
    static constexpr int OWN = SH::SRT * SH::SCG * 32;             // threads that hold S
    static constexpr int VEC = SH::SN / 8;                         // 16-byte vectors per thread
    static constexpr size_t BYTES = (size_t)(D * D + D) * sizeof(float);
    static_assert((size_t)OWN * VEC * 16 == (size_t)D * D * sizeof(float), "record");

    __device__ __forceinline__ static void write(uint8_t* rec, const State<T, D>& st, const float* zs) {
        if ((int)threadIdx.x < OWN) {
#pragma unroll
            for (int v = 0; v < VEC; ++v)
                reinterpret_cast<float4*>(rec)[v * OWN + threadIdx.x] = make_float4(st.S[v][0], st.S[v][1], st.S[v][2], st.S[v][3]);
        }
        float* z = reinterpret_cast<float*>(rec) + D * D;
        for (int a = threadIdx.x; a < D; a += SH::THREADS) z[a] = zs[a];
    }
    // Asks for the next chunk's record (d = 128, where no other CTA covers for the
    // wait: 2 % of the sweep; nothing gained at d = 64, fp32 loses 2 of 20).
    __device__ __forceinline__ static void ahead(const uint8_t* rec) {
        if constexpr (D == 128) {
            for (int a = threadIdx.x * 128; a < (int)BYTES; a += SH::THREADS * 128) prefetch_l2(rec + a);
        }
    }
    // this thread's part of <S, G> + <z, h>
    __device__ __forceinline__ static float product(const uint8_t* rec, const State<T, D>& st, const float* zs) {
        float sum = 0.f;
        if ((int)threadIdx.x < OWN) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const uint4 u = ldg_stream(reinterpret_cast<const uint4*>(rec) + v * OWN + threadIdx.x);
                sum += __uint_as_float(u.x) * st.S[v][0] + __uint_as_float(u.y) * st.S[v][1] +
                       __uint_as_float(u.z) * st.S[v][2] + __uint_as_float(u.w) * st.S[v][3];
            }
        }
        const float* z = reinterpret_cast<const float*>(rec) + D * D;
        for (int a = threadIdx.x; a < D; a += SH::THREADS) sum += z[a] * zs[a];
        return sum;
    }
};

template <typename T> __device__ __forceinline__ void load_pair(const T* p, float& a, float& b);
template <> __device__ __forceinline__ void load_pair<float>(const float* p, float& a, float& b) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    a = x.x;
    b = x.y;
}
template <> __device__ __forceinline__ void load_pair<__nv_bfloat16>(const __nv_bfloat16* p, float& a, float& b) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
    a = bf16_lo(x);
    b = bf16_hi(x);
}
__device__ __forceinline__ void store_pair(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(a, b);
}

// First sweep. 4x16x8192x64 bf16: 234 us for 336 MB of rows and 136 MB of chunk
// states (2.0 TB/s), fp32 660 us; 1x16x32768x128 bf16, identity: 494 us, 9.5 us
// for a chunk of 64 tokens. A chunk's products follow from one another over four
// barriers, and registers and shared memory leave an SM 8 warps at d = 128 (12 at 64)
// to cover for it: shared memory 62 % busy, the tensor pipe 33 %, issue 27 %.
template <typename T, int D, int PHI>
__global__ void __launch_bounds__(Shape<T, D>::THREADS, D == 64 ? 3 : 1)
gated_bwd_q_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                   const uint8_t* __restrict__ gates, const T* __restrict__ dout, const float* prefix, int N, int block_tokens, int nblk, int normalize,
                   T* __restrict__ dq, float* __restrict__ up, float* __restrict__ col, float* __restrict__ own, float* __restrict__ dgp,
                   uint8_t* __restrict__ chunk_state) {
    using SH = Shape<T, D>;
    using BQ = BwdQ<T, D, PHI>;
    constexpr int C = SH::C, LD = SH::LD, NT = SH::NCOL / 8;
    constexpr bool LO = BQ::PARTS == 2, APART = !SH::F32 && PHI == PHI_RELU1;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<typename BQ::Smem*>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    const int blk = blockIdx.x, bh = blockIdx.y;
    const int first = blk * block_tokens, end = min(N, first + block_tokens);
    const int nch = (end - first + C - 1) / C;
    const size_t off = (size_t)bh * N * D, toff = (size_t)bh * N;
    q += off; k += off; v += off; dout += off; dq += off;
    gates += ((size_t)bh * ((N + C - 1) / C) + first / C) * kGateBytes<C>;
    dgp += toff;
    uint8_t* states = chunk_state + ((size_t)bh * ((N + C - 1) / C) + first / C) * ChunkState<T, D>::BYTES;
    pdl_wait();

    auto fetch = [&](int c) {
        const int row0 = first + c * C;
        load_gates<C>(sm.gates[c & 1], gates + (size_t)c * kGateBytes<C>, nullptr, nullptr, nullptr, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][0], q, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][1], k, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][2], v, row0, N);
        load_tile<SH, T, D>(sm.tiles[c % SH::ST][3], dout, row0, N);
        cp_async_commit();
    };
    fetch(0);
    State<T, D> st;
    const float* rec = prefix ? prefix + ((size_t)bh * nblk + blk) * (size_t)(D * D + D) : nullptr;
    st.seed(rec, rec + D * D, warp, lane);
    st.template publish<LO>(sm.sop[0][0], sm.zs[0], warp, lane, sm.sop[0][BQ::PARTS - 1]);
    const int rg = row_group<SH>(warp), cg = warp / SH::RG;
    const int i0 = rg * 16, col0 = cg * SH::NCOL;

    // dgp of chunk c from the sums its warps left: a suffix sum over the chunk
    auto finish = [&](int c) {
        if (rg != 0 || cg != 0) return;  // a warp with one key group
        constexpr int R = C / 32;
        float x[R], run = 0.f;
#pragma unroll
        for (int e = R - 1; e >= 0; --e) {
            const int i = lane * R + e;
            x[e] = sm.row[c & 1][0][i] + run;
            run = x[e];
        }
        float after = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_down_sync(0xffffffffu, after, o);
            if (lane + o < 32) after += y;
        }
        after -= run;  // the lanes behind this one
#pragma unroll
        for (int e = 0; e < R; ++e) {
            const int i = first + c * C + lane * R + e;
            if (i < end) dgp[i] = x[e] + after;
        }
    };

    for (int c = 0; c < nch; ++c) {
        cp_async_wait<0>();
        __syncthreads();
        if (SH::ST == 2 && c + 1 < nch) fetch(c + 1);
        if (c > 0) finish(c - 1);
        const T *qt = sm.tiles[c % SH::ST][0], *kt = sm.tiles[c % SH::ST][1], *vt = sm.tiles[c % SH::ST][2], *gt = sm.tiles[c % SH::ST][3];
        const Gates<C>& gs = sm.gates[c & 1];
        const int sb = BQ::COPIES == 2 ? (c & 1) : 0;
        const T* sop = sm.sop[sb][0];
        const float* zs = sm.zs[sb];
        ChunkState<T, D>::write(states + (size_t)c * ChunkState<T, D>::BYTES, st, zs);

        // dout S^T, and q . z
        using PD = PhiDot<D, PHI>;
        float acc[NT][4] = {}, oz[4] = {}, sq[4] = {};
#pragma unroll(SH::F32 ? 1 : D / 16)
        for (int k0 = 0; k0 < D; k0 += 16) {
            FragA<T> a;
            load_a<LD>(a, gt, i0, k0, lane);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                FragB<T> b[2];
                load_bt<LD>(b, sop, col0 + 16 * n, k0, lane);
                mma_step(acc[2 * n], a, b[0]);
                mma_step(acc[2 * n + 1], a, b[1]);
                if constexpr (LO) {
                    load_bt<LD>(b, sm.sop[sb][1], col0 + 16 * n, k0, lane);
                    mma_step(acc[2 * n], a, b[0]);
                    mma_step(acc[2 * n + 1], a, b[1]);
                }
            }
            if (normalize || APART) {
                load_a<LD>(a, qt, i0, k0, lane);
                PD::rows(sq, a);
            }
            if (normalize) {
                FragB<T> b;
                load_column(b, zs, k0, lane);
                PD::column(oz, a, b);
            }
        }
        if (APART && normalize) {  // the ones' part, in column 0 like oz
            float sz = 0.f;
#pragma unroll
            for (int x = lane; x < D; x += 32) sz += zs[x];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sz += __shfl_xor_sync(0xffffffffu, sz, o);
            oz[0] += sz;
            oz[2] += sz;
        }
        // q . (S dout), over this warp's columns, then over the column groups
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x, y;
            const T* p = qt + (i0 + g) * LD + col0 + 8 * n + 2 * t;
            load_pair(p, x, y);
            s0 += phi_f<PHI>(x) * acc[n][0] + phi_f<PHI>(y) * acc[n][1];
            load_pair(p + 8 * LD, x, y);
            s1 += phi_f<PHI>(x) * acc[n][2] + phi_f<PHI>(y) * acc[n][3];
        }
        s0 = quad_sum(s0);
        s1 = quad_sum(s1);
        if constexpr (SH::CG > 1) {
            if (t == 0) {
                sm.part[cg][i0 + g] = s0;
                sm.part[cg][i0 + g + 8] = s1;
            }
            __syncthreads();
            s0 = s1 = 0.f;
#pragma unroll
            for (int x = 0; x < SH::CG; ++x) {
                s0 += sm.part[x][i0 + g];
                s1 += sm.part[x][i0 + g + 8];
            }
        }
        const bool deep = gs.deep;
        const float f0 = gs.from_start[i0 + g], f1 = gs.from_start[i0 + g + 8];
        const float hi0 = gs.hi[i0 + g], lo0 = gs.lo[i0 + g], hi1 = gs.hi[i0 + g + 8], lo1 = gs.lo[i0 + g + 8];
        // per row, over all keys in front: den = q . z and so on, num = sum of weights times dout . v
        float den0 = t == 0 ? f0 * (oz[0] + oz[1]) : 0.f, den1 = t == 0 ? f1 * (oz[2] + oz[3]) : 0.f;
        float num0 = 0.f, num1 = 0.f;
        float pd0 = 0.f, pd1 = 0.f, dd0 = 0.f, dd1 = 0.f;  // the own key's weight and dout . v
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            acc[n][0] *= f0; acc[n][1] *= f0; acc[n][2] *= f1; acc[n][3] *= f1;
        }
        float xs0 = 0.f, xs1 = 0.f, ys0 = 0.f, ys1 = 0.f;  // row sums of the operands below, for the shift of phi(k)
        float yk[NT][4] = {};
#pragma unroll 1
        for (int jt = 0; jt <= rg; ++jt) {
            float p[2][4], dp[2][4] = {};
            PD::template start<T>(p, sq);
#pragma unroll(SH::F32 ? 1 : D / 16)
            for (int k0 = 0; k0 < D; k0 += 16) {
                FragA<T> a;
                FragB<T> b[2];
                load_a<LD>(a, qt, i0, k0, lane);
                load_bt<LD>(b, kt, jt * 16, k0, lane);
                PD::step(p, a, b);
                load_a<LD>(a, gt, i0, k0, lane);
                load_bt<LD>(b, vt, jt * 16, k0, lane);
                mma_step(dp[0], a, b[0]);
                mma_step(dp[1], a, b[1]);
            }
            float w[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int jl = n * 8 + 2 * t, j = jt * 16 + jl;
                if (deep) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w[n][e] = decay(gs, hi0, lo0, j + e);
                        w[n][2 + e] = decay(gs, hi1, lo1, j + e);
                    }
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(gs.inv + j);
                    w[n][0] = f0 * x.x; w[n][1] = f0 * x.y; w[n][2] = f1 * x.x; w[n][3] = f1 * x.y;
                }
                if (jt == rg) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (jl + e == g) pd0 = p[n][e], dd0 = dp[n][e];
                        if (jl + e == g + 8) pd1 = p[n][2 + e], dd1 = dp[n][2 + e];
                        if (jl + e >= g) w[n][e] = 0.f;
                        if (jl + e >= g + 8) w[n][2 + e] = 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a0 = p[n][e] * w[n][e], a1 = p[n][2 + e] * w[n][2 + e];
                    den0 += a0;
                    den1 += a1;
                    num0 = fmaf(a0, dp[n][e], num0);
                    num1 = fmaf(a1, dp[n][2 + e], num1);
                    dp[n][e] *= w[n][e];
                    dp[n][2 + e] *= w[n][2 + e];
                    xs0 += dp[n][e];
                    xs1 += dp[n][2 + e];
                    ys0 += w[n][e];
                    ys1 += w[n][2 + e];
                }
            }
            // bf16: rounded once, like every operand of the gradients' products, but
            // for X under a positive map, from which delta Y is subtracted: that one
            // in two parts (dq at 2 x 8 x 4096 x 64, relu + 1: 3.0e-3 off with one)
            FragA<T> ax, xl, ay;
            {
                const float f[8] = {dp[0][0], dp[0][1], dp[0][2], dp[0][3], dp[1][0], dp[1][1], dp[1][2], dp[1][3]};
                split_a(ax, xl, f);
            }
            make_a(ay, w[0], w[1]);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                FragB<T> b[2];
                load_b<LD>(b, kt, jt * 16, col0 + 16 * n, lane);
                base_frag<PHI>(b[0]);
                base_frag<PHI>(b[1]);
                mma_step(acc[2 * n], ax, b[0]);
                mma_step(acc[2 * n + 1], ax, b[1]);
                if constexpr (LO && shifted<PHI>) {
                    mma_step(acc[2 * n], xl, b[0]);
                    mma_step(acc[2 * n + 1], xl, b[1]);
                }
                if (normalize) {
                    mma_step(yk[2 * n], ay, b[0]);
                    mma_step(yk[2 * n + 1], ay, b[1]);
                }
            }
        }
        den0 = quad_sum(den0);
        den1 = quad_sum(den1);
        // the state's part of num: q . (S dout)
        num0 = quad_sum(num0) + s0 * f0;
        num1 = quad_sum(num1) + s1 * f1;
        pd0 = quad_sum(pd0);
        pd1 = quad_sum(pd1);
        dd0 = quad_sum(dd0);
        dd1 = quad_sum(dd1);
        float up0 = 1.f, up1 = 1.f, de0 = 0.f, de1 = 0.f;
        // dd - de, and the row sum of W over the keys in front
        float df0 = dd0, df1 = dd1, rw0 = num0, rw1 = num1;
        const int row = first + c * C + i0 + g;
        if (normalize) {
            up0 = 1.f / (den0 + pd0);
            up1 = 1.f / (den1 + pd1);
            de0 = fmaf(pd0, dd0, num0) * up0;  // out . dout
            de1 = fmaf(pd1, dd1, num1) * up1;
            df0 = pd0 > den0 ? (dd0 * den0 - num0) * up0 : dd0 - de0;
            df1 = pd1 > den1 ? (dd1 * den1 - num1) * up1 : dd1 - de1;
            rw0 = -pd0 * up0 * df0;
            rw1 = -pd1 * up1 * df1;
            if (cg == 0 && t == 0) {
                if (row < end) {
                    up[toff + row] = up0;
                    col[toff + row] = -de0;
                    own[toff + row] = up0 * df0;
                }
                if (row + 8 < end) {
                    up[toff + row + 8] = up1;
                    col[toff + row + 8] = -de1;
                    own[toff + row + 8] = up1 * df1;
                }
            }
        }
        if (cg == 0 && t == 0) {
            sm.row[c & 1][0][i0 + g] = row < end ? rw0 : 0.f;
            sm.row[c & 1][0][i0 + g + 8] = row + 8 < end ? rw1 : 0.f;
        }
        xs0 = shifted<PHI> ? quad_sum(xs0) - de0 * quad_sum(ys0) : 0.f;
        xs1 = shifted<PHI> ? quad_sum(xs1) - de1 * quad_sum(ys1) : 0.f;
        const float dz0 = de0 * f0, dz1 = de1 * f1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x, y, kx, ky;
            const float2 z = *reinterpret_cast<const float2*>(zs + col0 + 8 * n + 2 * t);
            const int at = (i0 + g) * LD + col0 + 8 * n + 2 * t;
            const T *qp = qt + at, *kp = kt + at;
            T* o = dq + (size_t)row * D + col0 + 8 * n + 2 * t;
            if (row < end) {
                load_pair(qp, x, y);
                load_pair(kp, kx, ky);
                store_pair(o, up0 * (acc[n][0] + xs0 - de0 * yk[n][0] - dz0 * z.x + df0 * phi_f<PHI>(kx)) * slope_f<PHI>(x),
                           up0 * (acc[n][1] + xs0 - de0 * yk[n][1] - dz0 * z.y + df0 * phi_f<PHI>(ky)) * slope_f<PHI>(y));
            }
            if (row + 8 < end) {
                load_pair(qp + 8 * LD, x, y);
                load_pair(kp + 8 * LD, kx, ky);
                store_pair(o + 8 * D, up1 * (acc[n][2] + xs1 - de1 * yk[n][2] - dz1 * z.x + df1 * phi_f<PHI>(kx)) * slope_f<PHI>(x),
                           up1 * (acc[n][3] + xs1 - de1 * yk[n][3] - dz1 * z.y + df1 * phi_f<PHI>(ky)) * slope_f<PHI>(y));
            }
        }
        if (c + 1 < nch) {
            st.template update<PHI>(kt, vt, gs.to_end, nullptr, nullptr, true, gs.all, warp, lane);
            if (BQ::COPIES == 1) __syncthreads();  // every warp has read the operand and the tiles
            if (SH::ST == 1) fetch(c + 1);
            const int nb = BQ::COPIES == 2 ? ((c + 1) & 1) : 0;
            st.template publish<LO>(sm.sop[nb][0], sm.zs[nb], warp, lane, sm.sop[nb][BQ::PARTS - 1]);
        }
    }
    __syncthreads();
    finish(nch - 1);
}

// Second sweep, bound like the first. 4x16x8192x64 bf16: 235 us, fp32 744 us;
// 1x16x32768x128 bf16, identity: 541 us (shared memory 64 % busy, the tensor pipe 30 %).
template <typename T, int D, int PHI>
__global__ void __launch_bounds__(Shape<T, D>::THREADS, D == 64 ? 3 : 1)
gated_bwd_kv_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ gate,
                    const uint8_t* __restrict__ gates, const T* __restrict__ dout, const float* suffix, int N, int block_tokens, int nblk,
                    const float* up, const float* col, const float* own, const float* __restrict__ dgp,
                    const uint8_t* __restrict__ chunk_state, T* __restrict__ dk, T* __restrict__ dv, T* __restrict__ dg) {
    using SH = Shape<T, D>;
    constexpr int C = SH::C, LD = SH::LD, NT = SH::NCOL / 8;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<BwdKvSmem<T, D>*>(smem_raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane >> 2, t = lane & 3;
    const int blk = blockIdx.x, bh = blockIdx.y;
    const int first = blk * block_tokens, end = min(N, first + block_tokens);
    const int nch = (end - first + C - 1) / C;
    const size_t off = (size_t)bh * N * D, toff = (size_t)bh * N;
    q += off; k += off; v += off; dout += off; dk += off; dv += off;
    gate += toff;
    gates += ((size_t)bh * ((N + C - 1) / C) + first / C) * kGateBytes<C>;
    dgp += toff;
    dg += toff;
    if (up) {
        up += toff;
        col += toff;
        own += toff;
    }
    const uint8_t* states = chunk_state + ((size_t)bh * ((N + C - 1) / C) + first / C) * ChunkState<T, D>::BYTES;
    pdl_wait();

    // step s of the sweep is chunk nch - 1 - s
    auto fetch = [&](int s) {
        const int row0 = first + (nch - 1 - s) * C;
        load_gates<C>(sm.gates[s & 1], gates + (size_t)(nch - 1 - s) * kGateBytes<C>, up, col, own, row0, N);
        load_tile<SH, T, D>(sm.tiles[s % SH::ST][0], q, row0, N);
        load_tile<SH, T, D>(sm.tiles[s % SH::ST][1], k, row0, N);
        load_tile<SH, T, D>(sm.tiles[s % SH::ST][2], v, row0, N);
        load_tile<SH, T, D>(sm.tiles[s % SH::ST][3], dout, row0, N);
        cp_async_commit();
    };
    fetch(0);
    State<T, D> st;
    const float* rec = suffix ? suffix + ((size_t)bh * nblk + blk) * (size_t)(D * D + D) : nullptr;
    st.seed(rec, rec + D * D, warp, lane);
    st.publish(sm.sop[0][0], sm.zs[0], warp, lane);
    const int rg = row_group<SH>(warp), cg = warp / SH::RG;
    const int j0 = rg * 16, col0 = cg * SH::NCOL;

    // dg of step s: what the first sweep left, the keys in front and the outside
    auto finish = [&](int s) {
        // a warp with one query group (not a fixed one: 4x16x8192x128 622 us -> 597)
        if (rg != SH::RG - 1 || cg != 0) return;
        constexpr int R = C / 32;
        const int row0 = first + (nch - 1 - s) * C;
        float outside = 0.f;
#pragma unroll
        for (int w = 0; w < SH::NW; ++w) outside += sm.dot[s & 1][w];
        // sums over the keys in front of i, and over those from i on
        float x[R], w[R], own = 0.f, mine = 0.f;
#pragma unroll
        for (int e = 0; e < R; ++e) {
            const int i = lane * R + e;
            x[e] = own;
#pragma unroll
            for (int y = 0; y < SH::CG; ++y) own += sm.row[s & 1][y][i];
        }
#pragma unroll
        for (int e = R - 1; e >= 0; --e) {
            mine += sm.sum[s & 1][lane * R + e];
            w[e] = mine;
        }
        float run = own, after = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, run, o), z = __shfl_down_sync(0xffffffffu, after, o);
            if (lane >= o) run += y;
            if (lane + o < 32) after += z;
        }
        run -= own;
        after -= mine;
#pragma unroll
        for (int e = 0; e < R; ++e) {
            const int i = row0 + lane * R + e;
            if (i >= end) continue;
            // nothing passes a closed gate: its gradient is exactly 0
            const bool closed = to_f32<T>(gate[i]) < -104.f;  // e^g is 0 in fp32
            dg[i] = from_f32<T>(closed ? 0.f : (dgp[i] - (w[e] + after)) + (run + x[e]) + outside);
        }
    };

    for (int s = 0; s < nch; ++s) {
        const int c = nch - 1 - s;
        cp_async_wait<0>();
        __syncthreads();
        if (SH::ST == 2 && s + 1 < nch) fetch(s + 1);
        if (s + 1 < nch) ChunkState<T, D>::ahead(states + (size_t)(c - 1) * ChunkState<T, D>::BYTES);
        if (s > 0) finish(s - 1);
        const T *qt = sm.tiles[s % SH::ST][0], *kt = sm.tiles[s % SH::ST][1], *vt = sm.tiles[s % SH::ST][2], *gt = sm.tiles[s % SH::ST][3];
        const Gates<C>& gs = sm.gates[s & 1];
        const int sb = SH::SB == 2 ? (s & 1) : 0;
        const T* sop = sm.sop[sb][0];
        const float* zs = sm.zs[sb];

        float dot = gs.all * ChunkState<T, D>::product(states + (size_t)c * ChunkState<T, D>::BYTES, st, zs);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) sm.dot[s & 1][warp] = dot;

        // keys with the queries behind the chunk: phi(k) G and v G^T + h
        using PD = PhiDot<D, PHI>;
        float av[NT][4] = {}, ak[NT][4] = {}, sk[4] = {};
#pragma unroll(SH::F32 ? 1 : D / 16)
        for (int k0 = 0; k0 < D; k0 += 16) {
            FragA<T> a;
            FragB<T> b[2];
            load_a<LD>(a, kt, j0, k0, lane);
            PD::rows(sk, a);
            phi_frag<PHI>(a);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                load_b<LD>(b, sop, k0, col0 + 16 * n, lane);
                mma_step(av[2 * n], a, b[0]);
                mma_step(av[2 * n + 1], a, b[1]);
            }
            load_a<LD>(a, vt, j0, k0, lane);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                load_bt<LD>(b, sop, col0 + 16 * n, k0, lane);
                mma_step(ak[2 * n], a, b[0]);
                mma_step(ak[2 * n + 1], a, b[1]);
            }
        }
        const bool deep = gs.deep;
        const float e0 = gs.to_end[j0 + g], e1 = gs.to_end[j0 + g + 8];
        const float inv0 = gs.inv[j0 + g], inv1 = gs.inv[j0 + g + 8];
        const float own0 = up ? gs.own[j0 + g] : 0.f, own1 = up ? gs.own[j0 + g + 8] : 0.f;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float2 h = *reinterpret_cast<const float2*>(zs + col0 + 8 * n + 2 * t);
            av[n][0] *= e0; av[n][1] *= e0; av[n][2] *= e1; av[n][3] *= e1;
            ak[n][0] = e0 * (ak[n][0] + h.x);
            ak[n][1] = e0 * (ak[n][1] + h.y);
            ak[n][2] = e1 * (ak[n][2] + h.x);
            ak[n][3] = e1 * (ak[n][3] + h.y);
            float x, y;
            const T* p = kt + (j0 + g) * LD + col0 + 8 * n + 2 * t;
            load_pair(p, x, y);
            s0 += phi_f<PHI>(x) * ak[n][0] + phi_f<PHI>(y) * ak[n][1];
            load_pair(p + 8 * LD, x, y);
            s1 += phi_f<PHI>(x) * ak[n][2] + phi_f<PHI>(y) * ak[n][3];
        }
        s0 = quad_sum(s0);
        s1 = quad_sum(s1);
        const int row = first + c * C + j0 + g;
        if (t == 0) {  // a key past the last token holds nothing
            sm.row[s & 1][cg][j0 + g] = row < end ? s0 : 0.f;
            sm.row[s & 1][cg][j0 + g + 8] = row + 8 < end ? s1 : 0.f;
        }

        const float hi0 = gs.hi[j0 + g], lo0 = gs.lo[j0 + g], hi1 = gs.hi[j0 + g + 8], lo1 = gs.lo[j0 + g + 8];
        float rs0 = 0.f, rs1 = 0.f;  // row sums of the pairs' gradients, for the shift of phi(q)
        float ws0 = 0.f, ws1 = 0.f;  // row sums of W, own queries apart
#pragma unroll 1
        for (int it = rg; it < SH::RG; ++it) {
            float p[2][4], dp[2][4] = {};
            PD::template start<T>(p, sk);
#pragma unroll(SH::F32 ? 1 : D / 16)
            for (int k0 = 0; k0 < D; k0 += 16) {
                FragA<T> a;
                FragB<T> b[2];
                load_a<LD>(a, kt, j0, k0, lane);
                load_bt<LD>(b, qt, it * 16, k0, lane);
                PD::step(p, a, b);
                load_a<LD>(a, vt, j0, k0, lane);
                load_bt<LD>(b, gt, it * 16, k0, lane);
                mma_step(dp[0], a, b[0]);
                mma_step(dp[1], a, b[1]);
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int il = n * 8 + 2 * t, i = it * 16 + il;
                float2 cl = make_float2(0.f, 0.f);
                float w[4];
                if (deep) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w[e] = exp2_fast((gs.hi[i + e] - hi0) + (gs.lo[i + e] - lo0));
                        w[2 + e] = exp2_fast((gs.hi[i + e] - hi1) + (gs.lo[i + e] - lo1));
                    }
                } else {
                    const float2 f = *reinterpret_cast<const float2*>(gs.from_start + i);
                    w[0] = f.x * inv0; w[1] = f.y * inv0; w[2] = f.x * inv1; w[3] = f.y * inv1;
                }
                if (up) {
                    cl = *reinterpret_cast<const float2*>(gs.col + i);
                    const float2 u = *reinterpret_cast<const float2*>(gs.up + i);
                    w[0] *= u.x; w[1] *= u.y; w[2] *= u.x; w[3] *= u.y;
                }
                if (it == rg) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (il + e < g) w[e] = 0.f;
                        if (il + e < g + 8) w[2 + e] = 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool self = it == rg && il + (e & 1) == (e < 2 ? g : g + 8);  // the key's own query
                    dp[n][e] = w[e] * (dp[n][e] + (e & 1 ? cl.y : cl.x));
                    if (self && up) dp[n][e] = e < 2 ? own0 : own1;
                    (e < 2 ? ws0 : ws1) += self ? 0.f : p[n][e] * dp[n][e];
                    (e < 2 ? rs0 : rs1) += dp[n][e];
                    p[n][e] *= w[e];
                }
            }
            FragA<T> ap, ad;  // bf16: rounded once
            make_a(ap, p[0], p[1]);
            make_a(ad, dp[0], dp[1]);
#pragma unroll
            for (int n = 0; n < NT / 2; ++n) {
                FragB<T> b[2];
                load_b<LD>(b, gt, it * 16, col0 + 16 * n, lane);
                mma_step(av[2 * n], ap, b[0]);
                mma_step(av[2 * n + 1], ap, b[1]);
                load_b<LD>(b, qt, it * 16, col0 + 16 * n, lane);
                base_frag<PHI>(b[0]);
                base_frag<PHI>(b[1]);
                mma_step(ak[2 * n], ad, b[0]);
                mma_step(ak[2 * n + 1], ad, b[1]);
            }
        }
        if (cg == 0) {
            ws0 = quad_sum(ws0);
            ws1 = quad_sum(ws1);
            if (t == 0) {
                sm.sum[s & 1][j0 + g] = row < end ? ws0 : 0.f;
                sm.sum[s & 1][j0 + g + 8] = row + 8 < end ? ws1 : 0.f;
            }
        }
        rs0 = shifted<PHI> ? quad_sum(rs0) : 0.f;
        rs1 = shifted<PHI> ? quad_sum(rs1) : 0.f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float x, y;
            const int cc = col0 + 8 * n + 2 * t;
            const T* kp = kt + (j0 + g) * LD + cc;
            if (row < end) {
                load_pair(kp, x, y);
                store_pair(dk + (size_t)row * D + cc, (ak[n][0] + rs0) * slope_f<PHI>(x), (ak[n][1] + rs0) * slope_f<PHI>(y));
                store_pair(dv + (size_t)row * D + cc, av[n][0], av[n][1]);
            }
            if (row + 8 < end) {
                load_pair(kp + 8 * LD, x, y);
                store_pair(dk + (size_t)(row + 8) * D + cc, (ak[n][2] + rs1) * slope_f<PHI>(x), (ak[n][3] + rs1) * slope_f<PHI>(y));
                store_pair(dv + (size_t)(row + 8) * D + cc, av[n][2], av[n][3]);
            }
        }
        if (s + 1 < nch) {
            st.template update<PHI>(qt, gt, gs.from_start, up ? gs.up : nullptr, gs.col, up != nullptr, gs.all, warp, lane);
            if (SH::SB == 1) __syncthreads();  // every warp has read the operand and the tiles
            if (SH::ST == 1) fetch(s + 1);
            const int nb = SH::SB == 2 ? ((s + 1) & 1) : 0;
            st.publish(sm.sop[nb][0], sm.zs[nb], warp, lane);
        }
    }
    __syncthreads();
    finish(nch - 1);
}

template <typename T, int D, int PHI>
cudaError_t launch_bwd_q(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const void* dout,
                         const float* prefix, int block_tokens, int nblk, void* dq, float* up, float* col, float* own, float* dgp,
                         void* chunk_state, cudaStream_t st) {
    constexpr size_t smem = sizeof(typename BwdQ<T, D, PHI>::Smem);
    static_assert(smem <= 227 * 1024, "shared memory");
    const cudaError_t e = ensure_smem<gated_bwd_q_kernel<T, D, PHI>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(gated_bwd_q_kernel<T, D, PHI>, dim3((unsigned)nblk, (unsigned)p.bh()), dim3(Shape<T, D>::THREADS),
                      smem, st, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                      gates, static_cast<const T*>(dout), prefix, p.N, block_tokens, nblk,
                      p.normalize, static_cast<T*>(dq), up, col, own, dgp, static_cast<uint8_t*>(chunk_state));
}

template <typename T, int D, int PHI>
cudaError_t launch_bwd_kv(const Problem& p, const void* q, const void* k, const void* v, const void* g, const uint8_t* gates,
                          const void* dout, const float* suffix, int block_tokens, int nblk, const float* up, const float* col,
                          const float* own, const float* dgp, const void* chunk_state, void* dk, void* dv, void* dg, cudaStream_t st) {
    constexpr size_t smem = sizeof(BwdKvSmem<T, D>);
    static_assert(smem <= 227 * 1024, "shared memory");
    const cudaError_t e = ensure_smem<gated_bwd_kv_kernel<T, D, PHI>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(gated_bwd_kv_kernel<T, D, PHI>, dim3((unsigned)nblk, (unsigned)p.bh()), dim3(Shape<T, D>::THREADS),
                      smem, st, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                      static_cast<const T*>(g), gates, static_cast<const T*>(dout), suffix, p.N, block_tokens, nblk, up, col, own, dgp,
                      static_cast<const uint8_t*>(chunk_state), static_cast<T*>(dk), static_cast<T*>(dv),
                      static_cast<T*>(dg));
}

}  // namespace gated

template <typename T>
cudaError_t gated_bwd_q_t(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const void* dout,
                          const float* prefix, int block_tokens, int nblk, void* dq, float* up, float* col, float* own, float* dgp,
                          void* chunk_state, cudaStream_t st) {
    return gated::dispatch(p, [&](auto d, auto phi) {
        return gated::launch_bwd_q<T, decltype(d)::value, decltype(phi)::value>(
            p, q, k, v, gates, dout, prefix, block_tokens, nblk, dq, up, col, own, dgp, chunk_state, st);
    });
}
template <typename T>
cudaError_t gated_bwd_kv_t(const Problem& p, const void* q, const void* k, const void* v, const void* g, const uint8_t* gates,
                           const void* dout, const float* suffix, int block_tokens, int nblk, const float* up, const float* col,
                           const float* own, const float* dgp, const void* chunk_state, void* dk, void* dv, void* dg, cudaStream_t st) {
    return gated::dispatch(p, [&](auto d, auto phi) {
        return gated::launch_bwd_kv<T, decltype(d)::value, decltype(phi)::value>(
            p, q, k, v, g, gates, dout, suffix, block_tokens, nblk, up, col, own, dgp, chunk_state, dk, dv, dg, st);
    });
}

}  // namespace la
