// Gated linear attention at d = 128 on tcgen05 tensor cores (bf16), forward.
//
// Block states (tc_gated_state_kernel): a block's own state is
//   S = sum_j w_j phi(k_j) (x) v_j,  w_j = product of the block's gates behind j,
// with the weights relative to the block's end: the chunks run from the last
// to the first, so w is a running product and S is never rescaled. w phi(K) is
// formed in fp32 and multiplied as two bf16 operands (error 2^-17 of a term), or
// three for a state that the caller gets (none).
//
// Sweep (tc_gated_sweep_kernel): the transposed layout of the ungated d = 128
// sweep (tc_sweep_t.cu): S^T and O^T have d_v = 128 lanes. Per chunk, with
// b_i = log2 of the product of the chunk's gates up to i:
//   Q'   = 2^(n_i) phi(Q),  n_i = b_i rounded to a whole number within [-60, 0], or 0 (below)
//   O^T  = S_prev^T Q'^T
//   O^T += V^T P~^T,  P~_ij = (q'_i.phi(k_j)) 2^(-b_j)   j <= i
//   out_i = 2^(b_i - n_i) O_i / den_i,  den_i likewise (q'_i.z_prev + sum_j P~_ij)
//   S^T  = 2^(b_last) S^T + V^T (w phi(K)),  w_j = 2^(b_last - b_j)
// so that one accumulator takes both parts and the decay of a weight is one
// factor per key (and of a normalized output none at all). 2^(n_i) costs no
// bits of phi(q) and keeps what 2^(-b_j) multiplies as small as the decay makes
// the weight: without it products of some 2^37 left fp32. A chunk whose b all
// lie above -16 has no such factors and keeps n_i = 0, which spares the identity
// map its pass over Q (1x16x131072x128: sweep 467 us with the pass in every
// chunk, 433 - 440 with the choice; the other maps pass over Q anyway). Where b_i < -60,
// P~_ij = (q'_i.phi(k_j)) 2^(b_i + 60 - b_j), which leaves the state in front a
// weight of 2^(-60) next to the query's own key instead of the smaller true one
// (at 2^(-90) features below 2^(-36) would leave bf16's normal range).

#include "tc_gated.cuh"

namespace la {
namespace {

using namespace tcg;

// ---------------------------------------------------------------------------
// Block states
// ---------------------------------------------------------------------------
struct GsCfg {
    static constexpr int D = 128, C = 64, NB = 2, BOX = C * 128, TILE = NB * BOX;
    static constexpr int STAGES = 4;
    static constexpr int STAGE = 2 * TILE;          // K (becomes the high part), V
    static constexpr int PREP = 512, RED = PREP / 32 * D * 4;
    static constexpr int NBAR = 3 * STAGES + 2;
    static constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + 4 * TILE + RED + STAGES * 2 * C * 4 + 8 * NBAR + 16;
    static constexpr int THREADS = 64 + PREP;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Warp 0: TMA and gates; warp 1: MMA; warps 2..17: w phi(K) in its parts, z, and
// the accumulators' sums: the products of 8 chunks, or 4 for a state that the
// caller gets, are added to fp32 registers, so long blocks do not depend on how
// the tensor core rounds its additions (S at 1x16x16384x128: 3.4e-7 off with 2
// chunks, 6.9e-7 with 4, over 1e-6 with 8; 1x16x131072x128 takes 283, 257, 246 us).
// REVERSE (gradients): K = q, V = dout, chunks in order, weights the product of
// the block's gates up to the query times up_i = 1 / den_i, and z weighted by
// col_i = -(out_i . dout_i); without up and col (not normalized) 1 and 0.
template <int PHI, bool REVERSE>
__global__ void __launch_bounds__(GsCfg::THREADS, 1)
tc_gated_state_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                      const __nv_bfloat16* __restrict__ gate, const float* __restrict__ up, const float* __restrict__ col,
                      int N, int block_tokens, int nblk, int blk0, int exact, float* __restrict__ part, float* __restrict__ dec, uint32_t* __restrict__ err) {
    using CF = GsCfg;
    constexpr int D = CF::D, C = CF::C;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stages = align1024(smem_raw);
    uint8_t* lo = stages + CF::STAGES * CF::STAGE;  // low parts of two chunks, then their last bits
    float* red = reinterpret_cast<float*>(lo + 4 * CF::TILE);
    float* wts = red + CF::RED / 4;  // [stage][weights C | of z C]
    uint64_t* full = reinterpret_cast<uint64_t*>(wts + CF::STAGES * 2 * C);
    uint64_t* tdone = full + CF::STAGES;
    uint64_t* empty = tdone + CF::STAGES;
    uint64_t* acc = empty + CF::STAGES;  // [2] accumulator complete
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc + 2);
    const int warp = warp_index(), lane = threadIdx.x % 32;
    const int blk = blk0 + blockIdx.x, bh = blockIdx.y;
    const int first = blk * block_tokens, end = min(N, first + block_tokens);
    const int nci = (end - first + C - 1) / C;
    const int per = exact ? 2 : 3;  // log2 of the chunks per accumulation
    if (threadIdx.x == 0) {
        cta_abort_reset();
        for (int s = 0; s < CF::STAGES; ++s) {
            mbar_init(full + s, 1);
            mbar_init(tdone + s, CF::PREP / 32);
            mbar_init(empty + s, 1);
        }
        mbar_init(acc, 1);
        mbar_init(acc + 1, 1);
        fence_mbar_init();
        tma_prefetch_map(&mK);
        tma_prefetch_map(&mV);
    }
    if (warp == 1) tmem_alloc(tmem_slot, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    // step i is chunk nci - 1 - i, or i
    auto row_of = [&](int i) { return first + (REVERSE ? i : nci - 1 - i) * C; };
    if (warp == 0) {
        const __nv_bfloat16* g = gate + (size_t)bh * N;
        long long after = 0;  // the block's gates behind the chunk, or in front of it
        bool bad = false;
        Gates2 gr = load_gates(g, row_of(0), end, lane);
        float2 ur = make_float2(1.f, 1.f), cr = make_float2(0.f, 0.f);
        auto load_sums = [&](int row) {
            if (!REVERSE || up == nullptr) return;
            const size_t at = (size_t)bh * N + row + 2 * lane;
            const bool in0 = row + 2 * lane < end, in1 = row + 2 * lane + 1 < end;
            ur = make_float2(in0 ? up[at] : 0.f, in1 ? up[at + 1] : 0.f);
            cr = make_float2(in0 ? col[at] : 0.f, in1 ? col[at + 1] : 0.f);
        };
        load_sums(row_of(0));
        int issued = 0;
#pragma unroll 1
        for (int i = 0; i < nci; ++i) {
            const int s = i % CF::STAGES, u = i / CF::STAGES, row = row_of(i);
            const GateSums<2> gs = sum_gates<2>(gr.g, lane);
            bad = bad || gs.bad & 4;
            if (i + 1 < nci) gr = load_gates(g, row_of(i + 1), end, lane);
            const float2 un = ur, cn = cr;
            if (i + 1 < nci) load_sums(row_of(i + 1));
            if (u > 0 && !__all_sync(0xffffffffu, mbar_wait(empty + s, (u - 1) & 1, err))) break;
            float* w = wts + s * 2 * C + 2 * lane;
            const float nan = bad ? NAN : 0.f;  // the block's state is NaN
            const bool in0 = row + 2 * lane < end, in1 = row + 2 * lane + 1 < end;
            if (REVERSE) {
                w[0] = in0 ? gate_pow2(after + gs.b[0]) * un.x + nan : 0.f;
                w[1] = in1 ? gate_pow2(after + gs.b[1]) * un.y + nan : 0.f;
                w[C] = cn.x;
                w[C + 1] = cn.y;
            } else {
                w[0] = in0 ? gate_pow2(after + (gs.last - gs.b[0])) + nan : 0.f;
                w[1] = in1 ? gate_pow2(after + (gs.last - gs.b[1])) + nan : 0.f;
            }
            after = gate_add(after, gs.last);
            __syncwarp();
            if (elect_one()) {
                mbar_arrive_expect_tx(full + s, CF::STAGE);
                uint8_t* st = stages + s * CF::STAGE;
#pragma unroll
                for (int bx = 0; bx < CF::NB; ++bx) {
                    tma_load_3d(st + bx * CF::BOX, &mK, full + s, bx * 64, row, bh);
                    tma_load_3d(st + CF::TILE + bx * CF::BOX, &mV, full + s, bx * 64, row, bh);
                }
            }
            __syncwarp();
            issued = i + 1;
        }
        if (lane == 0) {
            dec[(size_t)bh * nblk + blk] = gate_pow2(after) + (bad ? NAN : 0.f);
            for (int i = max(0, issued - CF::STAGES); i < issued; ++i)
                mbar_wait(full + i % CF::STAGES, (i / CF::STAGES) & 1, err, false);
        }
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_bf16(D, D, true, true);
        const uint64_t kd = sdesc(smem_u32(stages), CF::BOX, 1024), ld = sdesc(smem_u32(lo), CF::BOX, 1024);
#pragma unroll 1
        for (int i = 0; i < nci; ++i) {
            const int s = i % CF::STAGES, f = i >> per;
            if (!__all_sync(0xffffffffu, mbar_wait(tdone + s, (i / CF::STAGES) & 1, err))) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t k0 = kd + s * (CF::STAGE >> 4), v0 = k0 + (CF::TILE >> 4), l0 = ld + (i & 1) * (CF::TILE >> 4);
                const uint32_t d = tmem + (f & 1) * D;
                uint32_t add = i & ((1 << per) - 1) ? 1u : 0u;
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk) {  // 16 tokens: 16 rows of 128 bytes
                    if (exact) {
                        mma_bf16(d, l0 + 2 * (CF::TILE >> 4) + kk * 128, v0 + kk * 128, id, add);
                        add = 1u;
                    }
                    mma_bf16(d, l0 + kk * 128, v0 + kk * 128, id, add);
                    add = 1u;
                    mma_bf16(d, k0 + kk * 128, v0 + kk * 128, id, 1u);
                }
                mma_commit(empty + s);
                if (i + 1 == nci || ((i + 1) & ((1 << per) - 1)) == 0) mma_commit(acc + (f & 1));
            }
            __syncwarp();
        }
    } else {
        const int et = threadIdx.x - 64, wq = warp - 2, sp = warp & 3, quarter = wq / 4;
        const uint32_t lane_base = static_cast<uint32_t>(sp * 32) << 16;
        const int g = (lane & 7) ^ ((et >> 3) & 7);  // column group (of 8) of this thread's 16-byte chunks
        float S[32], zk[CF::NB][8];
#pragma unroll
        for (int e = 0; e < 32; ++e) S[e] = 0.f;
#pragma unroll
        for (int b = 0; b < CF::NB; ++b)
#pragma unroll
            for (int e = 0; e < 8; ++e) zk[b][e] = 0.f;
        // adds accumulator f; its next use starts two flushes later, behind
        // the tdone arrivals of every thread here
        auto take = [&](int f) {
            mbar_wait(acc + (f & 1), (f >> 1) & 1, err);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t r[16];
                tmem_ld16(tmem + lane_base + (f & 1) * D + quarter * 32 + 16 * c, r);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) S[16 * c + e] += __uint_as_float(r[e]);
            }
            tc_fence_before();
        };
#pragma unroll 1
        for (int i = 0;; ++i) {
            const int s = i % CF::STAGES, u = i / CF::STAGES;
            // accumulator f is taken during the first chunk of flush f + 1, or at the end
            if (i > 0 && (i == nci || (i & ((1 << per) - 1)) == 0)) take((i - 1) >> per);
            if (i == nci) break;
            mbar_wait(full + s, u & 1, err);
            // the low part's buffer: chunk i - 2's products have read it
            if (i >= 2) mbar_wait(empty + (i - 2) % CF::STAGES, ((i - 2) / CF::STAGES) & 1, err);
            uint8_t* kt = stages + s * CF::STAGE;
            uint8_t* lt = lo + (i & 1) * CF::TILE;
            const float* w = wts + s * 2 * C;
            const float zw = REVERSE ? w[C + (et >> 3)] : 1.f;
#pragma unroll
            for (int bx = 0; bx < CF::NB; ++bx) {  // each thread one 16-byte chunk per box: token et >> 3
                uint4* kp = reinterpret_cast<uint4*>(kt + bx * CF::BOX + et * 16);
                float f[8];
                uint4 phi, hi, rest;
                weighted8<PHI>(*kp, w[et >> 3], f, phi, hi, rest);
                *kp = hi;
                *reinterpret_cast<uint4*>(lt + bx * CF::BOX + et * 16) = rest;
                if (exact) {  // a state that the caller gets keeps all bits of w phi(K)
                    float a[8], b[8];
                    unpack8(hi, a);
                    unpack8(rest, b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] = (f[e] - a[e]) - b[e];
                    *reinterpret_cast<uint4*>(lt + 2 * CF::TILE + bx * CF::BOX + et * 16) = pack8(a);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) zk[bx][e] = REVERSE ? fmaf(f[e], zw, zk[bx][e]) : zk[bx][e] + f[e];
            }
            fence_async_smem();
            tc_fence_before();
            warp_arrive(tdone + s, lane);
        }
        float* rec = part + ((size_t)bh * nblk + blk) * (size_t)(D * D + D);
#pragma unroll
        for (int bx = 0; bx < CF::NB; ++bx) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // lanes l, l^9, l^18, l^27 hold the same column group
                zk[bx][e] += __shfl_xor_sync(0xffffffffu, zk[bx][e], 9);
                zk[bx][e] += __shfl_xor_sync(0xffffffffu, zk[bx][e], 18);
            }
            if (lane < 8) {
                float4* dst = reinterpret_cast<float4*>(red + wq * D + bx * 64 + g * 8);
                dst[0] = make_float4(zk[bx][0], zk[bx][1], zk[bx][2], zk[bx][3]);
                dst[1] = make_float4(zk[bx][4], zk[bx][5], zk[bx][6], zk[bx][7]);
            }
        }
        named_bar(1, CF::PREP);
        if (et < D) {
            float z = 0.f;
#pragma unroll
            for (int x = 0; x < CF::PREP / 32; ++x) z += red[x * D + et];
            rec[(size_t)D * D + et] = z;
        }
        float4* o = reinterpret_cast<float4*>(rec + (size_t)(sp * 32 + lane) * D + quarter * 32);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ---------------------------------------------------------------------------
// Sweep
// ---------------------------------------------------------------------------
// Warp roles (704 threads): warp 0 TMA and gates, warp 1 MMA and TMEM, warps
// 2..9 "transform" (phi on K, w phi(K) in two parts, z), warps 10..13
// "state" (phi on Q; S^T: the bf16 operand, and its decay in place), warps 14..17 "mask"
// (P~, denominators), warps 18..21 "out" (O^T to the outputs). The transforms run a chunk ahead: the loop
// from one S^T update to the next holds only the state warps' pass over S^T
// and that update's products. 1x16x131072x128, relu + 1: 463 us for 2147 MB, 4.6
// TB/s, 71 % of a copy's rate; the rest is that loop, about 3,900 cycles a chunk.
struct GtCfg {
    static constexpr int D = 128, C = 64, NB = 2;
    static constexpr int BOX = C * 128;            // one 64-row x 64-column box (8 KB)
    static constexpr int KBOX = (C + 16) * 128;    // K box + 16 rows: z_prev in 8 parts, high and low
    static constexpr int TILE = NB * BOX;
    static constexpr int QK = TILE + NB * KBOX;    // Q, K' of a chunk: two slots, free after its P and O^T
    static constexpr int VS = 3;                   // V slots: free after its O^T += V^T P~^T, a chunk later
    static constexpr int GS = 4;                   // gate slots [b | 2^-b | 2^n twice, bf16 | what fp32 left of b]
    static constexpr int PT = C * C * 2;           // P~ [query][key], K-major (x2)
    static constexpr int STG = TILE;               // output staging tile
    static constexpr int KW = 2 * TILE;            // w phi(K), high and low part (x2)
    static constexpr int INV = 2 * C * 4;          // output scale per query row (x2)
    static constexpr int GATES = GS * 4 * C * 4;
    static constexpr int NBAR = 2 + 2 + 2 * VS + GS + 2 + 2 + 2 + 5 * 2;
    static constexpr size_t SMEM = 1024 + 2 * (size_t)QK + VS * TILE + 2 * PT + STG + 2 * KW + INV + GATES +
                                   8 * NBAR + 16;
    // TMEM columns, as in tc_sweep_t.cu
    static constexpr int COL_S = 0, COL_SB = 128, COL_P = 256, COL_O = 384;
    static constexpr int TRANSFORM = 256, STATE = 128, MASK = 128, OUT = 128;
    static constexpr int THREADS = 64 + TRANSFORM + STATE + MASK + OUT;
    static constexpr int AHEAD = 4;                // chunks between a prefetch into L2 and the load
    static_assert(SMEM + 16 <= 227 * 1024, "shared memory (16 bytes static)");
    static_assert(QK % 1024 == 0 && KBOX % 1024 == 0, "1024-byte aligned operand tiles");
};

template <int PHI>
__global__ void __launch_bounds__(GtCfg::THREADS, 1)
tc_gated_sweep_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                      const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mOut,
                      const __nv_bfloat16* __restrict__ gate, const float* __restrict__ prefix,
                      const float* __restrict__ S_in, const float* __restrict__ z_in, int N, int block_tokens, int nblk,
                      int normalize, uint32_t* __restrict__ err) {
    using CF = GtCfg;
    constexpr int D = CF::D, C = CF::C;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* qks = align1024(smem_raw);
    uint8_t* vs = qks + 2 * CF::QK;
    uint8_t* pt = vs + CF::VS * CF::TILE;
    uint8_t* stg = pt + 2 * CF::PT;
    uint8_t* kws = stg + CF::STG;
    float* inv = reinterpret_cast<float*>(kws + 2 * CF::KW);
    float* gates = inv + 2 * C;
    uint64_t* fullqk = reinterpret_cast<uint64_t*>(gates + CF::GS * 4 * C);
    uint64_t* emptyqk = fullqk + 2;
    uint64_t* fullv = emptyqk + 2;
    uint64_t* emptyv = fullv + CF::VS;
    uint64_t* gfull = emptyv + CF::VS;     // gates of a chunk written
    uint64_t* bstate = gfull + CF::GS;     // Q and the S_prev^T operand written, S^T scaled
    uint64_t* bsdone = bstate + 1;         // S^T update of the chunk done
    uint64_t* btrans = bsdone + 1;         // per slot (chunk % 2): K' and w phi(K) written
    uint64_t* kwfree = btrans + 2;         // w phi(K) read
    uint64_t* bpfull = kwfree + 2;         // P ready, P~ written, O^T ready, O^T read
    uint64_t* bptready = bpfull + 2;
    uint64_t* bofull = bptready + 2;
    uint64_t* bofree = bofull + 2;
    uint64_t* binv = bofree + 2;           // output scales written
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(binv + 2);

    const int warp = warp_index(), lane = threadIdx.x % 32;
    const int blk = blockIdx.x, bh = blockIdx.y;
    const int first = blk * block_tokens, end = min(N, first + block_tokens);
    const int nci = (end - first + C - 1) / C;

    if (threadIdx.x == 0) {
        cta_abort_reset();
        for (int j = 0; j < CF::VS; ++j) {
            mbar_init(fullv + j, 1);
            mbar_init(emptyv + j, 1);
        }
        for (int j = 0; j < CF::GS; ++j) mbar_init(gfull + j, 1);
        mbar_init(bstate, CF::STATE / 32);
        mbar_init(bsdone, 1);
        for (int j = 0; j < 2; ++j) {
            mbar_init(fullqk + j, 1);
            mbar_init(emptyqk + j, 1);
            mbar_init(btrans + j, CF::TRANSFORM / 32);
            mbar_init(kwfree + j, 1);
            mbar_init(bpfull + j, 1);
            mbar_init(bptready + j, CF::MASK / 32);
            mbar_init(bofull + j, 1);
            mbar_init(bofree + j, CF::OUT / 32);
            mbar_init(binv + j, CF::MASK / 32);
        }
        fence_mbar_init();
        tma_prefetch_map(&mQ);
        tma_prefetch_map(&mK);
        tma_prefetch_map(&mV);
        tma_prefetch_map(&mOut);
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    if (warp == 0) {
        // ---------------- TMA producer and gates (whole warp) ----------------
        const __nv_bfloat16* g = gate + (size_t)bh * N;
        Gates2 gr = load_gates(g, first, end, lane);
        int nqk = 0, nv = 0;
#pragma unroll 1
        for (int ci = 0; ci < nci; ++ci) {
            const int j = ci & 1, s = ci % CF::VS, row = first + ci * C;
            const GateSums<2> sums = sum_gates<2>(gr.g, lane);
            if (ci + 1 < nci) gr = load_gates(g, row + C, end, lane);
            // in two floats: behind closed gates (14000 bits each) one would not
            // hold what lies between two tokens
            const float2 b0 = gate_float2(sums.b[0]), b1 = gate_float2(sums.b[1]);
            const float f0 = b0.x + (sums.bad & 1 ? NAN : 0.f), f1 = b1.x + (sums.bad & 2 ? NAN : 0.f);
            const bool low = __any_sync(0xffffffffu, fminf(f0, f1) < kDeep);
            const bool steep = __any_sync(0xffffffffu, fminf(f0, f1) < kSteep);
            // 2^-b, or in its first place infinity: some query lies below kDeep
            const float2 inv2 = make_float2(lane == 0 && low ? INFINITY : ex2(-f0), ex2(-f1));
            const float2 pow2 = make_float2(__uint_as_float(whole_pow2(f0, steep)), __uint_as_float(whole_pow2(f1, steep)));
            // chunk ci - 2's P and O^T are done, and with them (in order) all
            // that chunk ci - 4 needed its gates for
            if (ci >= 2 && !__all_sync(0xffffffffu, mbar_wait(emptyqk + j, ((ci >> 1) - 1) & 1, err))) break;
            float2* gs = reinterpret_cast<float2*>(gates + (ci % CF::GS) * 4 * C) + lane;
            gs[0] = make_float2(f0, f1);
            gs[C / 2] = inv2;
            gs[C] = pow2;
            gs[3 * C / 2] = make_float2(b0.y, b1.y);
            __syncwarp();
            if (elect_one()) {
                mbar_arrive(gfull + ci % CF::GS);
                mbar_arrive_expect_tx(fullqk + j, 2 * CF::TILE);
                uint8_t* st = qks + j * CF::QK;
#pragma unroll
                for (int bx = 0; bx < CF::NB; ++bx) {
                    tma_load_3d(st + CF::TILE + bx * CF::KBOX, &mK, fullqk + j, bx * 64, row, bh);
                    tma_load_3d(st + bx * CF::BOX, &mQ, fullqk + j, bx * 64, row, bh);
                }
            }
            __syncwarp();
            nqk = ci + 1;
            if (ci >= CF::VS && !__all_sync(0xffffffffu, mbar_wait(emptyv + s, (ci / CF::VS - 1) & 1, err))) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(fullv + s, CF::TILE);
#pragma unroll
                for (int bx = 0; bx < CF::NB; ++bx)
                    tma_load_3d(vs + s * CF::TILE + bx * CF::BOX, &mV, fullv + s, bx * 64, row, bh);
                if (ci + CF::AHEAD < nci) {
#pragma unroll
                    for (int bx = 0; bx < CF::NB; ++bx) {
                        tma_prefetch_3d(&mK, bx * 64, row + CF::AHEAD * C, bh);
                        tma_prefetch_3d(&mQ, bx * 64, row + CF::AHEAD * C, bh);
                        tma_prefetch_3d(&mV, bx * 64, row + CF::AHEAD * C, bh);
                    }
                }
            }
            __syncwarp();
            nv = ci + 1;
        }
        // drain: the loads still in flight land before the CTA exits
        if (lane == 0) {
            for (int c = max(0, nqk - 2); c < nqk; ++c) mbar_wait(fullqk + (c & 1), (c >> 1) & 1, err, false);
            for (int c = max(0, nv - CF::VS); c < nv; ++c)
                mbar_wait(fullv + c % CF::VS, (c / CF::VS) & 1, err, false);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (whole warp; one lane issues) ----------------
        const uint32_t idP = idesc_bf16(C, normalize ? C + 16 : C, false, false);  // P = Q [K; z]^T
        constexpr uint32_t idS = idesc_bf16(D, D, true, true);    // S^T += V^T (w K)
        constexpr uint32_t idO = idesc_bf16(D, C, false, false);  // O^T = S_prev^T Q^T
        constexpr uint32_t idV = idesc_bf16(D, C, true, false);   // O^T += V^T P~^T
        const uint64_t dq0 = sdesc(smem_u32(qks), 16, 1024), dk0 = dq0 + (CF::TILE >> 4);
        const uint64_t dv0 = sdesc(smem_u32(vs), CF::BOX, 1024), dw0 = sdesc(smem_u32(kws), CF::BOX, 1024);
        const uint64_t dp0 = sdesc(smem_u32(pt), 16, 1024);
        bool ok = true;
        // O^T += V^T P~^T of chunk `ci`, issued after the next chunk's P and O^T
        auto flush = [&](int ci) {
            const int j = ci & 1;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bptready + j, (ci >> 1) & 1, err));
            if (!ok) return;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t v = dv0 + (ci % CF::VS) * (CF::TILE >> 4), pp = dp0 + j * (CF::PT >> 4);
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    mma_bf16(tmem + CF::COL_O + j * C, v + kk * 128, pp + kk * 2, idV, 1u);
                mma_commit(bofull + j);
                mma_commit(emptyv + ci % CF::VS);
            }
            __syncwarp();
        };
#pragma unroll 1
        for (int ci = 0; ci <= nci; ++ci) {
            const int j = ci & 1, k = ci >> 1;
            if (ci < nci) {
                const uint64_t q = dq0 + j * (CF::QK >> 4), kd = dk0 + j * (CF::QK >> 4);
                ok = mbar_wait(fullv + ci % CF::VS, (ci / CF::VS) & 1, err) && mbar_wait(btrans + j, k & 1, err) &&
                     mbar_wait(bstate, ci & 1, err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t v = dv0 + (ci % CF::VS) * (CF::TILE >> 4), w = dw0 + j * (CF::KW >> 4);
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        mma_bf16(tmem + CF::COL_S, v + kk * 128, w + (CF::TILE >> 4) + kk * 128, idS, 1u);
                        mma_bf16(tmem + CF::COL_S, v + kk * 128, w + kk * 128, idS, 1u);
                    }
                    mma_commit(bsdone);
                    mma_commit(kwfree + j);
                    // P[j] was read two chunks ago (that chunk's P~ was waited for in its flush)
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_bf16(tmem + CF::COL_P + j * (16u << 16), q + (kk / 4) * (CF::BOX >> 4) + (kk % 4) * 2,
                                 kd + (kk / 4) * (CF::KBOX >> 4) + (kk % 4) * 2, idP, kk > 0);
                    mma_commit(bpfull + j);
                }
                __syncwarp();
                if (k > 0) ok = __all_sync(0xffffffffu, mbar_wait(bofree + j, (k - 1) & 1, err));  // O^T[j] read two chunks ago
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sb = tmem + CF::COL_SB + j * 64;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_bf16_ts(tmem + CF::COL_O + j * C, sb + kk * 8, q + (kk / 4) * (CF::BOX >> 4) + (kk % 4) * 2, idO,
                                    kk > 0);
                    mma_commit(emptyqk + j);
                }
                __syncwarp();
            }
            if (ci > 0) flush(ci - 1);
        }
    } else if (warp < 10) {
        // ---------------- transform warps ----------------
        const int et = threadIdx.x - 64, wq = warp - 2;
        const float* pz = prefix ? prefix + ((size_t)bh * nblk + blk) * (size_t)(D * D + D) + D * D
                          : z_in ? z_in + (size_t)bh * D
                                 : nullptr;
        const int g = (lane & 7) ^ ((et >> 3) & 7);  // column group (of 8) of this thread's 16-byte chunks
        // z_prev stands in 8 parts, one per warp (the tokens that warp transforms
        // in every chunk): row 64 + wq of the K boxes is the part's bf16 value,
        // row 72 + wq the rounding remainder, and P's columns 64..79 add up to
        // phi(Q).z_prev. The lanes l, l^9, l^18, l^27 hold the same column group
        // g of both boxes; each keeps two of its columns, from column zc on.
        const int zc = 8 * g + 4 * ((lane >> 3) & 1) + 2 * (lane >> 4);
        float2 zp[CF::NB];
#pragma unroll
        for (int bx = 0; bx < CF::NB; ++bx)
            zp[bx] = pz && wq == 0 ? make_float2(pz[bx * 64 + zc], pz[bx * 64 + zc + 1]) : make_float2(0.f, 0.f);
#pragma unroll 1
        for (int ci = 0; ci < nci; ++ci) {
            const int j = ci & 1, k = ci >> 1;
            const int kvalid = min(C, end - first - ci * C);
            uint8_t* kt = qks + j * CF::QK + CF::TILE;
            uint8_t* kw = kws + j * CF::KW;
            mbar_wait(fullqk + j, k & 1, err);
            const float* gs = gates + (ci % CF::GS) * 4 * C;
            const float blast = gs[C - 1], rest = gs[4 * C - 1];
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = (et >> 3) + 32 * i;
                w[i] = r < kvalid ? ex2((blast - gs[r]) + (rest - gs[3 * C + r])) : 0.f;
            }
            const float all = ex2(blast);
            if (k > 0) mbar_wait(kwfree + j, (k - 1) & 1, err);  // chunk ci - 2's update has read kw
#pragma unroll
            for (int bx = 0; bx < CF::NB; ++bx) {
                float cs[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) cs[e] = 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int p = et + 256 * i;  // 16-byte chunk within the box (token (et >> 3) + 32 i)
                    uint4* kp = reinterpret_cast<uint4*>(kt + bx * CF::KBOX + p * 16);
                    float f[8];
                    uint4 phi, hi, lo;
                    weighted8<PHI>(*kp, w[i], f, phi, hi, lo);
                    *reinterpret_cast<uint4*>(kw + bx * CF::BOX + p * 16) = hi;
                    *reinterpret_cast<uint4*>(kw + CF::TILE + bx * CF::BOX + p * 16) = lo;
                    if (PHI != PHI_IDENTITY) *kp = phi;  // rows past the end are masked in P~
#pragma unroll
                    for (int e = 0; e < 8; ++e) cs[e] += f[e];
                }
                if (normalize) {
                    const uint32_t hi = pack_bf16(zp[bx].x, zp[bx].y);
                    const float2 rest = make_float2(zp[bx].x - __uint_as_float(hi << 16),
                                                    zp[bx].y - __uint_as_float(hi & 0xffff0000u));
                    uint8_t* kb = kt + bx * CF::KBOX;
                    *reinterpret_cast<uint32_t*>(kb + sw128_off(C + wq, zc)) = hi;
                    *reinterpret_cast<uint32_t*>(kb + sw128_off(C + 8 + wq, zc)) = pack_bf16(rest.x, rest.y);
                    // the warp's column sums: lanes with bit 3 set keep columns
                    // 4..7 of the group, then lanes with bit 4 set the upper two
                    float s4[4], s2[2];
                    const bool b3 = lane & 8, b4 = lane & 16;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float give = b3 ? cs[e] : cs[4 + e], keep = b3 ? cs[4 + e] : cs[e];
                        s4[e] = keep + __shfl_xor_sync(0xffffffffu, give, 9);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float give = b4 ? s4[e] : s4[2 + e], keep = b4 ? s4[2 + e] : s4[e];
                        s2[e] = keep + __shfl_xor_sync(0xffffffffu, give, 18);
                    }
                    zp[bx].x = fmaf(zp[bx].x, all, s2[0]);
                    zp[bx].y = fmaf(zp[bx].y, all, s2[1]);
                }
            }
            fence_async_smem();
            warp_arrive(btrans + j, lane);
        }
    } else if (warp < 14) {
        // ---------------- state warps ----------------
        const int sp = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(sp * 32) << 16;
        const int a = sp * 32 + lane;  // the S^T row (d_v) of this thread
        const float* pS = prefix ? prefix + ((size_t)bh * nblk + blk) * (size_t)(D * D + D)
                          : S_in ? S_in + (size_t)bh * D * D
                                 : nullptr;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t r[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = pS ? __float_as_uint(pS[(size_t)(c0 + e) * D + a]) : 0u;
            tmem_st16(tmem + CF::COL_S + lane_base + c0, r);
        }
        tmem_st_wait();
#pragma unroll 1
        for (int ci = 0; ci < nci; ++ci) {
            const int et = threadIdx.x - (64 + CF::TRANSFORM);
            const float* gs = gates + (ci % CF::GS) * 4 * C;
            mbar_wait(gfull + ci % CF::GS, (ci / CF::GS) & 1, err);
            const float all = ex2(gs[C - 1]);
            // phi on the chunk's queries and their scales, while the last update runs
            const uint32_t* pow2 = reinterpret_cast<const uint32_t*>(gs + 2 * C);
            if (PHI != PHI_IDENTITY || __any_sync(0xffffffffu, pow2[lane] != kOne2 || pow2[lane + 32] != kOne2)) {
                mbar_wait(fullqk + (ci & 1), (ci >> 1) & 1, err);
                uint4* q = reinterpret_cast<uint4*>(qks + (ci & 1) * CF::QK);
#pragma unroll 2
                for (int x = et; x < CF::TILE / 16; x += CF::STATE)  // 8 pieces of 16 bytes per row of a box
                    q[x] = scale8(phi_round8<PHI>(q[x]), pow2[(x / 8) % C]);
                fence_async_smem();
            }
            if (ci > 0) {
                mbar_wait(bsdone, (ci - 1) & 1, err);
                tc_fence_after();
            }
            // S_prev^T -> bf16 pairs, and scaled in place for this chunk's update
            const uint32_t sb = tmem + CF::COL_SB + (ci & 1) * 64 + lane_base;
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
                const uint32_t col = tmem + CF::COL_S + lane_base + 32 * h;
                uint32_t r[32];
                tmem_ld16(col, *reinterpret_cast<uint32_t(*)[16]>(r));
                tmem_ld16(col + 16, *reinterpret_cast<uint32_t(*)[16]>(r + 16));
                tmem_ld_wait();
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack_bf16(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
                tmem_st16(sb + 16 * h, w);
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * all);
                tmem_st16(col, *reinterpret_cast<uint32_t(*)[16]>(r));
                tmem_st16(col + 16, *reinterpret_cast<uint32_t(*)[16]>(r + 16));
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(bstate, lane);
        }
    } else if (warp < 18) {
        // ---------------- mask warps ----------------
        const int sp = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(sp * 32) << 16;
        const int i = sp * 16 + (lane & 15);  // P row (query) of this thread: M = 64 layout
        const int half = lane >= 16 ? 1 : 0;  // the two warp halves take the two column halves
#pragma unroll 1
        for (int ci = 0; ci < nci; ++ci) {
            const int slot = ci & 1, use = ci >> 1;
            const uint32_t lane_s = lane_base + static_cast<uint32_t>(slot) * (16u << 16);
            uint8_t* pts = pt + slot * CF::PT;
            mbar_wait(gfull + ci % CF::GS, (ci / CF::GS) & 1, err);
            const float* gs = gates + (ci % CF::GS) * 4 * C;
            const float bi = gs[i];
            const bool deep = isinf(gs[C]);  // some query of the chunk lies below kDeep
            mbar_wait(bpfull + slot, use & 1, err);
            tc_fence_after();
            uint32_t r[32], zq[8];
            tmem_ld16x2<32>(tmem + CF::COL_P + lane_s, *reinterpret_cast<uint32_t(*)[16]>(r));
            tmem_ld16x2<32>(tmem + CF::COL_P + lane_s + 16, *reinterpret_cast<uint32_t(*)[16]>(r + 16));
            if (normalize) tmem_ld8x2<8>(tmem + CF::COL_P + lane_s + C, zq);
            tmem_ld_wait();
            if (deep) {  // the factors per pair, from both floats; the table's are not used then
                const bool below = bi < kDeep;
                const float hi = below ? bi : 0.f, lo = below ? gs[3 * C + i] : 0.f, up = below ? -kDeep : 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const int j = 32 * half + e;
                    r[e] = __float_as_uint(__uint_as_float(r[e]) * ex2((hi - gs[j]) + (lo - gs[3 * C + j]) + up));
                }
            }
            float rs = 0.f;
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
                float f[8];
                const int j0 = 32 * half + 8 * gq;
                const float4 x = *reinterpret_cast<const float4*>(gs + C + j0);
                const float4 y = *reinterpret_cast<const float4*>(gs + C + j0 + 4);
                const float e8[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = j0 + e <= i ? __uint_as_float(r[8 * gq + e]) * (deep ? 1.f : e8[e]) : 0.f;
                const uint4 w = pack8(f);
                *reinterpret_cast<uint4*>(pts + sw128_off(i, j0)) = w;
                // the denominator sums the rounded weights: the output is a mean with these very weights
                unpack8(w, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) rs += f[e];
            }
            fence_async_smem();
            tc_fence_before();
            warp_arrive(bptready + slot, lane);
            if (normalize) {
#pragma unroll
                for (int e = 0; e < 8; ++e) rs += __uint_as_float(zq[e]);  // phi(Q_i).z_prev, half of its parts
                rs += __shfl_xor_sync(0xffffffffu, rs, 16);
            }
            // the scales of chunk ci - 2 have been read
            if (use > 0) mbar_wait(bofree + slot, (use - 1) & 1, err);
            if (lane < 16) inv[slot * C + i] = normalize ? __frcp_rn(rs) : ex2(fmaxf(bi, kDeep) - whole_bits(__float_as_uint(gs[2 * C + i])));
            warp_arrive(binv + slot, lane);
        }
    } else {
        // ---------------- out warps ----------------
        const int sp = warp & 3, et = threadIdx.x - (CF::THREADS - CF::OUT);
        const int mi = lane >> 3, mj = lane & 7, q2 = 2 * (lane & 3);
        const uint32_t stg_u = smem_u32(stg);
        bool ok = true;  // no early exit (named barrier 3); a failed wait only suppresses the stores
#pragma unroll 1
        for (int ci = 0; ci < nci; ++ci) {
            const int slot = ci & 1, use = ci >> 1;
            const float* scale = inv + slot * C;
            ok = mbar_wait(binv + slot, use & 1, err) && ok;
            ok = mbar_wait(bofull + slot, use & 1, err) && ok;
            tc_fence_after();
            if (et == 0) bulk_wait_read0();  // the previous chunk's store has read stg
            named_bar(3, CF::OUT);
            // O^T rows (d_v) a0 .. a0 + 15, 16 columns (queries) at a time: the
            // 16x256b TMEM shape hands each lane the fragment that stmatrix .trans
            // stores with the queries as rows
#pragma unroll 1
            for (int hl = 0; hl < 2; ++hl) {
                const int a0 = sp * 32 + 16 * hl;
                uint32_t o[32];
                tmem_ld16x256_x8(tmem + CF::COL_O + slot * C + (static_cast<uint32_t>(a0) << 16), o);
                tmem_ld_wait();
                const uint32_t box = stg_u + (a0 / 64) * CF::BOX;
                const int ch = (a0 % 64) / 8 + (mi & 1);
#pragma unroll
                for (int cb = 0; cb < C; cb += 16) {
                    const float2 i0 = *reinterpret_cast<const float2*>(scale + cb + q2);
                    const float2 i1 = *reinterpret_cast<const float2*>(scale + cb + 8 + q2);
                    const uint32_t* x = o + (cb / 8) * 4;
                    const uint32_t p0 = pack_bf16(__uint_as_float(x[0]) * i0.x, __uint_as_float(x[1]) * i0.y);
                    const uint32_t p1 = pack_bf16(__uint_as_float(x[2]) * i0.x, __uint_as_float(x[3]) * i0.y);
                    const uint32_t p2 = pack_bf16(__uint_as_float(x[4]) * i1.x, __uint_as_float(x[5]) * i1.y);
                    const uint32_t p3 = pack_bf16(__uint_as_float(x[6]) * i1.x, __uint_as_float(x[7]) * i1.y);
                    const uint32_t row = cb + 8 * (mi >> 1) + mj;
                    stmatrix_x4_trans(box + row * 128u + ((static_cast<uint32_t>(ch) ^ (row & 7u)) << 4), p0, p1, p2, p3);
                }
            }
            tc_fence_before();
            warp_arrive(bofree + slot, lane);  // O^T[slot] and its scales read
            fence_async_smem();
            named_bar(3, CF::OUT);
            if (et == 0 && ok) {
#pragma unroll
                for (int bx = 0; bx < CF::NB; ++bx) tma_store_3d(&mOut, stg + bx * CF::BOX, bx * 64, first + ci * C, bh);
                bulk_commit();
            }
        }
        if (et == 0) bulk_wait0();  // the output stores have landed
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int PHI, bool REVERSE>
cudaError_t launch_state(const Problem& p, const void* k, const void* v, const void* g, const float* up, const float* col,
                         int block_tokens, int nblk, int blk0, int count, bool exact, float* part, float* dec, uint32_t* err, cudaStream_t st) {
    using CF = GsCfg;
    CUtensorMap mk, mv;
    cudaError_t e = make_map(&mk, k, CF::D, p.N, p.bh(), CF::C);
    if (e == cudaSuccess) e = make_map(&mv, v, CF::D, p.N, p.bh(), CF::C);
    if (e == cudaSuccess) e = ensure_smem<tc_gated_state_kernel<PHI, REVERSE>>(CF::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(tc_gated_state_kernel<PHI, REVERSE>, dim3((unsigned)count, (unsigned)p.bh()), dim3(CF::THREADS), CF::SMEM, st,
                      mk, mv, static_cast<const __nv_bfloat16*>(g), up, col, p.N, block_tokens, nblk, blk0, (int)exact, part, dec,
                      err);
}

template <int PHI>
cudaError_t launch_sweep(const Problem& p, const void* q, const void* k, const void* v, const void* g, const float* prefix,
                         const float* S_in, const float* z_in, int block_tokens, int nblk, void* out, uint32_t* err,
                         cudaStream_t st) {
    using CF = GtCfg;
    CUtensorMap mq, mk, mv, mo;
    cudaError_t e = make_map(&mq, q, CF::D, p.N, p.bh(), CF::C);
    if (e == cudaSuccess) e = make_map(&mk, k, CF::D, p.N, p.bh(), CF::C);
    if (e == cudaSuccess) e = make_map(&mv, v, CF::D, p.N, p.bh(), CF::C);
    if (e == cudaSuccess) e = make_map(&mo, out, CF::D, p.N, p.bh(), CF::C);
    if (e == cudaSuccess) e = ensure_smem<tc_gated_sweep_kernel<PHI>>(CF::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl(tc_gated_sweep_kernel<PHI>, dim3((unsigned)nblk, (unsigned)p.bh()), dim3(CF::THREADS), CF::SMEM, st,
                      mq, mk, mv, mo, static_cast<const __nv_bfloat16*>(g), prefix, S_in, z_in, p.N, block_tokens, nblk,
                      p.normalize, err);
}

}  // namespace

bool tc_gated_supported(const Problem& p) { return p.dtype == DT_BF16 && p.d == 128; }

cudaError_t tc_gated_states(const Problem& p, bool reverse, const void* x, const void* y, const void* g, const float* up,
                            const float* col, int block_tokens, int nblk, int blk0, int count, bool exact, float* part,
                            float* dec, uint32_t* err, cudaStream_t st) {
    auto* f = reverse ? (p.phi == PHI_RELU1  ? launch_state<PHI_RELU1, true>
                         : p.phi == PHI_ELU1 ? launch_state<PHI_ELU1, true>
                                             : launch_state<PHI_IDENTITY, true>)
                      : (p.phi == PHI_RELU1  ? launch_state<PHI_RELU1, false>
                         : p.phi == PHI_ELU1 ? launch_state<PHI_ELU1, false>
                                             : launch_state<PHI_IDENTITY, false>);
    return f(p, x, y, g, up, col, block_tokens, nblk, blk0, count, exact, part, dec, err, st);
}

cudaError_t tc_gated_sweep(const Problem& p, const void* q, const void* k, const void* v, const void* g,
                           const float* prefix, const float* S_in, const float* z_in, int block_tokens, int nblk, void* out,
                           uint32_t* err, cudaStream_t st) {
    auto* f = p.phi == PHI_RELU1  ? launch_sweep<PHI_RELU1>
              : p.phi == PHI_ELU1 ? launch_sweep<PHI_ELU1>
                                  : launch_sweep<PHI_IDENTITY>;
    return f(p, q, k, v, g, prefix, S_in, z_in, block_tokens, nblk, out, err, st);
}

}  // namespace la
