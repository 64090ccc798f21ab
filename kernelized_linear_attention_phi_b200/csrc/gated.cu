// Gated linear attention: the scan of block states, the one-token step and
// the choice of the element type's kernels (gated_bf16.cu, gated_f32.cu).

#include "gate_scan.cuh"
#include "gated.h"
#include "gated_common.cuh"
#include "launch_util.h"

namespace la {
namespace {

// The gates of every chunk of C tokens, as the sweeps take them (a warp per
// chunk): once per call, so that no sweep waits for a scan between two chunks.
// Little more than its launch (7 us for 16 rows of 4096, 11 for 64 of 8192).
template <typename T, int C>
__global__ void __launch_bounds__(128) gates_kernel(const T* __restrict__ gate, int N, int nch, uint8_t* __restrict__ out) {
    using namespace gated;
    constexpr int R = C / 32;
    using Raw = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
    const int c = blockIdx.x * 4 + threadIdx.x / 32, lane = threadIdx.x % 32, bh = blockIdx.y;
    pdl_wait();
    if (c >= nch) return;
    const Raw* g = reinterpret_cast<const Raw*>(gate) + (size_t)bh * N;
    Raw raw[R];
#pragma unroll
    for (int e = 0; e < R; ++e) {
        const int i = c * C + lane * R + e;
        raw[e] = i < N ? g[i] : Raw(0);
    }
    const GateSums<R> q = sum_gates<R>(raw, lane);
    Gates<C>& s = *reinterpret_cast<Gates<C>*>(out + ((size_t)bh * nch + c) * kGateBytes<C>);
    bool low = false;
    const float whole = q.bad >> R ? NAN : 0.f;
#pragma unroll
    for (int e = 0; e < R; ++e) {
        const int i = lane * R + e;
        const float nan = q.bad & (1 << e) ? NAN : 0.f;
        const float2 b = gate_float2(q.b[e]);
        const bool in = c * C + i < N;
        low = low || !(fabsf(b.x) <= kDeep);
        s.hi[i] = b.x + nan;
        s.lo[i] = b.y;
        s.from_start[i] = in ? gate_pow2(q.b[e]) + nan : 0.f;
        s.inv[i] = gate_pow2(-q.b[e]) + nan;
        s.to_end[i] = in ? gate_pow2(q.last - q.b[e]) + whole : 0.f;
    }
    low = __any_sync(0xffffffffu, low);
    if (lane == 0) {
        s.all = gate_pow2(q.last) + whole;
        s.deep = low;
    }
}

template <typename T, int C>
cudaError_t launch_gates(const Problem& p, const void* g, uint8_t* out, cudaStream_t st) {
    const int nch = (p.N + C - 1) / C;
    return launch_pdl(gates_kernel<T, C>, dim3((unsigned)((nch + 3) / 4), (unsigned)p.bh()), dim3(128), 0, st,
                      static_cast<const T*>(g), p.N, nch, out);
}

// Record blk of each head becomes the state in front of the block (REVERSE:
// behind it), from S_in / z_in or zero; the state past the other end goes to
// S_out / z_out. One thread per entry of the state, its records' loads in flight
// together; S_out may be S_in. Bound by launch and two round trips: 8 - 14 us.
template <bool REVERSE>
__global__ void __launch_bounds__(256)
gated_scan_kernel(float* __restrict__ rec, const float* __restrict__ dec, int nblk, int dd, int sf, const float* S_in,
                  const float* z_in, float* S_out, float* z_out) {
    const int e = blockIdx.x * 256 + threadIdx.x, bh = blockIdx.y;
    pdl_wait();
    if (e >= sf) return;
    const size_t si = (size_t)bh * dd + e, zi = (size_t)bh * (sf - dd) + e - dd;
    float run = 0.f;
    if (S_in) run = e < dd ? S_in[si] : z_in[zi];
    float* r = rec + (size_t)bh * nblk * sf + e;
    const float* w = dec + (size_t)bh * nblk;
    const bool last = S_out != nullptr;
    constexpr int U = 8;  // records in flight
    for (int b0 = 0; b0 < nblk; b0 += U) {
        float own[U], a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int b = REVERSE ? nblk - 1 - (b0 + u) : b0 + u;
            const bool in = b0 + u < nblk && (last || b0 + u + 1 < nblk);
            own[u] = in ? r[(size_t)b * sf] : 0.f;
            a[u] = in ? w[b] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b0 + u >= nblk) break;
            const int b = REVERSE ? nblk - 1 - (b0 + u) : b0 + u;
            r[(size_t)b * sf] = run;
            run = fmaf(a[u], run, own[u]);
        }
    }
    if (last) {
        if (e < dd) S_out[si] = run;
        else z_out[zi] = run;
    }
}

// One token on a cached state, every (b, h) at once: a CTA per head streams the
// d x d state through registers once (bandwidth bound: 2 d (d + 1) fp32 moved
// per head and step, nothing else of note). The state's loads are issued
// before the token's rows are needed, so one round trip covers both.
// 64x32 heads of 128: 43.4 us for 273 MB, 6.3 TB/s, 96 % of a copy's rate.
constexpr int kThreads = 256;

__device__ __forceinline__ float4 ld_cs(const float4* p) {
    float4 r;
    asm volatile("ld.global.cs.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ void st_cs(float4* p, float4 v) {
    asm volatile("st.global.cs.v4.f32 [%0], {%1,%2,%3,%4};" ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// phi_apply, but a NaN with its sign set stays one too.
__device__ __forceinline__ float phi_step(float x, int phi) {
    return phi == PHI_RELU1 ? relu_nan(x) + 1.f : phi_apply(x, phi);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
gated_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ gate,
                    const float* S, const float* z, float* S_out, float* z_out, T* __restrict__ out, int phi, int normalize) {
    constexpr int NCG = D / 4;           // float4 column groups per row
    constexpr int NRG = kThreads / NCG;  // row groups
    constexpr int RPT = (D + NRG - 1) / NRG;
    __shared__ float spk[D], spq[D];
    __shared__ __align__(16) float sv[D], red[NRG][D];
    __shared__ float sden[kThreads / 32];
    const long long bh = blockIdx.x;
    const int tid = threadIdx.x, cg = tid % NCG, rg = tid / NCG;
    pdl_wait();
    const float4* Sh = reinterpret_cast<const float4*>(S + bh * (long long)D * D);
    float4* So = reinterpret_cast<float4*>(S_out + bh * (long long)D * D);
    float4 s[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int a = rg + r * NRG;
        if (a < D) s[r] = ld_cs(Sh + a * NCG + cg);
    }
    const float decay = expf(to_f32<T>(gate[bh]));
    float dpart = 0.f;
    if (tid < D) {
        const float zo = z[bh * D + tid];
        const float pk = phi_step(to_f32<T>(k[bh * D + tid]), phi), pq = phi_step(to_f32<T>(q[bh * D + tid]), phi);
        spk[tid] = pk;
        spq[tid] = pq;
        sv[tid] = to_f32<T>(v[bh * D + tid]);
        const float zn = fmaf(decay, zo, pk);
        z_out[bh * D + tid] = zn;
        dpart = pq * zn;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dpart += __shfl_xor_sync(0xffffffffu, dpart, o);
    if ((tid & 31) == 0) sden[tid >> 5] = dpart;
    __syncthreads();
    const float4 vv = *reinterpret_cast<const float4*>(sv + cg * 4);
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const int a = rg + r * NRG;
        if (a < D) {
            const float pk = spk[a], pq = spq[a];
            s[r].x = fmaf(decay, s[r].x, pk * vv.x);
            s[r].y = fmaf(decay, s[r].y, pk * vv.y);
            s[r].z = fmaf(decay, s[r].z, pk * vv.z);
            s[r].w = fmaf(decay, s[r].w, pk * vv.w);
            st_cs(So + a * NCG + cg, s[r]);
            num.x = fmaf(pq, s[r].x, num.x);
            num.y = fmaf(pq, s[r].y, num.y);
            num.z = fmaf(pq, s[r].z, num.z);
            num.w = fmaf(pq, s[r].w, num.w);
        }
    }
    if (rg < NRG) *reinterpret_cast<float4*>(&red[rg][cg * 4]) = num;
    __syncthreads();
    if (tid < D) {
        float acc = 0.f;
#pragma unroll
        for (int r = 0; r < NRG; ++r) acc += red[r][tid];
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) den += sden[w];
        out[bh * D + tid] = from_f32<T>(normalize ? acc / den : acc);
    }
}

template <typename T, int D>
cudaError_t launch_decode(const Problem& p, const void* q, const void* k, const void* v, const void* g, const float* S,
                          const float* z, float* S_out, float* z_out, void* out, cudaStream_t st) {
    return launch_pdl(gated_decode_kernel<T, D>, dim3((unsigned)p.bh()), dim3(kThreads), 0, st, static_cast<const T*>(q),
                      static_cast<const T*>(k), static_cast<const T*>(v), static_cast<const T*>(g), S, z, S_out, z_out,
                      static_cast<T*>(out), p.phi, p.normalize);
}

template <typename T>
cudaError_t decode_t(const Problem& p, const void* q, const void* k, const void* v, const void* g, const float* S,
                     const float* z, float* S_out, float* z_out, void* out, cudaStream_t st) {
    switch (p.d) {
        case 16: return launch_decode<T, 16>(p, q, k, v, g, S, z, S_out, z_out, out, st);
        case 32: return launch_decode<T, 32>(p, q, k, v, g, S, z, S_out, z_out, out, st);
        case 64: return launch_decode<T, 64>(p, q, k, v, g, S, z, S_out, z_out, out, st);
        case 128: return launch_decode<T, 128>(p, q, k, v, g, S, z, S_out, z_out, out, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t gated_decode(const Problem& p, const void* q, const void* k, const void* v, const void* g, const float* S,
                         const float* z, float* S_out, float* z_out, void* out, cudaStream_t st) {
    if (p.dtype == DT_F32) return decode_t<float>(p, q, k, v, g, S, z, S_out, z_out, out, st);
    return decode_t<__nv_bfloat16>(p, q, k, v, g, S, z, S_out, z_out, out, st);
}

cudaError_t gated_scan(const Problem& p, bool reverse, float* rec, const float* dec, int nblk, const float* S_in,
                       const float* z_in, float* S_out, float* z_out, cudaStream_t st) {
    const int dd = p.d * p.d, sf = (int)p.state_floats();
    const dim3 grid((unsigned)((sf + 255) / 256), (unsigned)p.bh());
    if (reverse)
        return launch_pdl(gated_scan_kernel<true>, grid, dim3(256), 0, st, rec, dec, nblk, dd, sf, S_in, z_in, S_out, z_out);
    return launch_pdl(gated_scan_kernel<false>, grid, dim3(256), 0, st, rec, dec, nblk, dd, sf, S_in, z_in, S_out, z_out);
}

cudaError_t gated_gates(const Problem& p, const void* g, uint8_t* out, cudaStream_t st) {
    if (p.dtype == DT_BF16) return launch_gates<__nv_bfloat16, 64>(p, g, out, st);
    return gated_chunk(p) == 32 ? launch_gates<float, 32>(p, g, out, st) : launch_gates<float, 64>(p, g, out, st);
}
size_t gated_gate_bytes(const Problem& p) {
    const size_t one = gated_chunk(p) == 32 ? gated::kGateBytes<32> : gated::kGateBytes<64>;
    return (size_t)p.bh() * ((p.N + gated_chunk(p) - 1) / gated_chunk(p)) * one;
}

// fp32 d >= 64: chunks of 32 tokens (gated_common.cuh, Shape)
int gated_chunk(const Problem& p) { return p.dtype == DT_F32 && p.d >= 64 ? 32 : 64; }
size_t gated_chunk_state_bytes(const Problem& p) {
    return p.state_floats() * sizeof(float);
}

cudaError_t gated_sweep(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const float* prefix,
                        const float* S_in, const float* z_in, int block_tokens, int nblk, void* out, float* S_out,
                        float* z_out, cudaStream_t st) {
    auto* f = p.dtype == DT_F32 ? gated_sweep_t<float> : gated_sweep_t<__nv_bfloat16>;
    return f(p, q, k, v, gates, prefix, S_in, z_in, block_tokens, nblk, out, S_out, z_out, st);
}
cudaError_t gated_states(const Problem& p, bool reverse, const void* x, const void* y, const uint8_t* gates, const float* up,
                         const float* col, int block_tokens, int nblk, int blk0, int count, bool exact, float* rec, float* dec,
                         cudaStream_t st) {
    auto* f = p.dtype == DT_F32 ? gated_states_t<float> : gated_states_t<__nv_bfloat16>;
    return f(p, reverse, x, y, gates, up, col, block_tokens, nblk, blk0, count, exact, rec, dec, st);
}
cudaError_t gated_bwd_q(const Problem& p, const void* q, const void* k, const void* v, const uint8_t* gates, const void* dout,
                        const float* prefix, int block_tokens, int nblk, void* dq, float* up, float* col, float* own, float* dgp,
                        void* chunk_state, cudaStream_t st) {
    auto* f = p.dtype == DT_F32 ? gated_bwd_q_t<float> : gated_bwd_q_t<__nv_bfloat16>;
    return f(p, q, k, v, gates, dout, prefix, block_tokens, nblk, dq, up, col, own, dgp, chunk_state, st);
}
cudaError_t gated_bwd_kv(const Problem& p, const void* q, const void* k, const void* v, const void* g, const uint8_t* gates, const void* dout,
                         const float* suffix, int block_tokens, int nblk, const float* up, const float* col,
                         const float* own, const float* dgp, const void* chunk_state, void* dk, void* dv, void* dg, cudaStream_t st) {
    auto* f = p.dtype == DT_F32 ? gated_bwd_kv_t<float> : gated_bwd_kv_t<__nv_bfloat16>;
    return f(p, q, k, v, g, gates, dout, suffix, block_tokens, nblk, up, col, own, dgp, chunk_state, dk, dv, dg, st);
}

}  // namespace la
