// Norm of every query and key row with the position rotation, one pass:
//   u = x * r * w,  r = (mean(x^2) + eps)^(-1/2),  y = R(position) u,
// R turning the channel pairs (i, i + rot/2), or (2i, 2i + 1), by the angles
// whose cosines and sines are row `position` of the tables; channels past rot
// pass through. Rows are read where a projection left them (any strides, the
// row itself contiguous) and written to [B, H, N, d].
//
// Backward, with n = x r and v = R^T dy (R is orthogonal on the pairs):
//   dw = sum v n,  dx = r (v w - n mean(v w n)).
//
// Bound by memory: a row is read and written once (backward: x, dy read, dx
// written), 16 bytes per lane, d / 8 (bf16) or d / 4 (fp32) lanes per row. The
// lanes of a token keep its cosines and sines in registers and run over
// several heads, so the tables (fp32, as wide as the rows) are read once per
// head group and not once per row. Forward, 4x16384x(16+16)x64 bf16: 95 us for
// 541 MB, 87 % of a copy's rate. Backward, 3x1777x(12+4)x128 fp32: 34 us for
// 132 MB (60 %); 2x4096x(8+8)x64 bf16: 23 us for 51 MB, of which some 6 are
// the launch; registers (two rows and the sums of dw) hold it to 5 CTAs an SM.

#include "common.cuh"
#include "device.h"
#include "launch_util.h"
#include "qk_rope.h"

namespace la {
namespace {

// Forward, small CTAs: tokens of many places in flight (4x16384x(16+16)x64 bf16:
// 104 us with 256 threads, 95 with 128; 105 with 8 rows in flight, for 97). Backward, larger ones: fewer rows of
// partial weight gradients.
constexpr int kForward = 128, kThreads = 256;
constexpr int kInFlight = 4;  // rows a lane loads before it uses the first

struct Side {  // queries or keys
    const void* x;
    const void* dy;
    void* y;           // forward: [B, H, N, d]; backward: dx by strides ys
    const float* w;
    la_strides xs, ys;
    int H, groups;     // heads, head groups of `per` heads
};
struct Args {
    Side s[2];
    const float *cos, *sin;
    const int32_t* positions;
    float* part;
    long long tokens;  // B * N
    int N, rot, rows, per;
    float eps;
};

// What a token's lanes hold: their channels' cosines and (signed) sines.
template <typename T, int D, bool PAIRS> struct Turn {
    static constexpr int EPV = Vec16<T>::N, LPR = D / EPV;
    float c[EPV], s[EPV];
    int partner;  // lane that holds the other channel of each pair (halves)
    bool bad;

    __device__ __forceinline__ void load(const Args& p, long long token, int l) {
        const int e0 = l * EPV, half = p.rot / 2, lane = threadIdx.x % 32;
        const int pos = p.positions ? p.positions[token] : (int)(token % p.N);
        bad = p.rot > 0 && (pos < 0 || pos >= p.rows);
        partner = lane;
#pragma unroll
        for (int e = 0; e < EPV; ++e) c[e] = 1.f, s[e] = 0.f;
        if (e0 >= p.rot || bad) return;
        const float* cr = p.cos + (size_t)pos * half;
        const float* sr = p.sin + (size_t)pos * half;
        if (PAIRS) {
#pragma unroll
            for (int e = 0; e < EPV; e += 2) {
                c[e] = c[e + 1] = cr[(e0 + e) / 2];
                s[e + 1] = sr[(e0 + e) / 2];
                s[e] = -s[e + 1];
            }
        } else {
            const bool low = e0 < half;
            const int i0 = low ? e0 : e0 - half;
            partner = low ? lane + half / EPV : lane - half / EPV;
#pragma unroll
            for (int e = 0; e < EPV; e += 4) {
                const float4 a = *reinterpret_cast<const float4*>(cr + i0 + e);
                const float4 b = *reinterpret_cast<const float4*>(sr + i0 + e);
                c[e] = a.x; c[e + 1] = a.y; c[e + 2] = a.z; c[e + 3] = a.w;
                s[e] = b.x; s[e + 1] = b.y; s[e + 2] = b.z; s[e + 3] = b.w;
            }
            if (low) {
#pragma unroll
                for (int e = 0; e < EPV; ++e) s[e] = -s[e];
            }
        }
    }
    // The pairs' other channels of a row as it was loaded (x its own, unpacked).
    // Every lane of the warp calls it.
    __device__ __forceinline__ void others(const uint4& raw, const float (&x)[EPV], float (&o)[EPV]) const {
        if constexpr (PAIRS) {
#pragma unroll
            for (int e = 0; e < EPV; ++e) o[e] = x[e ^ 1];
        } else {
            uint4 u;
            u.x = __shfl_sync(0xffffffffu, raw.x, partner);
            u.y = __shfl_sync(0xffffffffu, raw.y, partner);
            u.z = __shfl_sync(0xffffffffu, raw.z, partner);
            u.w = __shfl_sync(0xffffffffu, raw.w, partner);
            Vec16<T>::unpack(u, o);
        }
    }
};

template <int LPR> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kForward) qk_rope_kernel(const __grid_constant__ Args p) {
    using TU = Turn<T, D, PAIRS>;
    constexpr int EPV = TU::EPV, LPR = TU::LPR, RPB = kForward / LPR;
    const int l = threadIdx.x % LPR;
    const int which = (int)blockIdx.y >= p.s[0].groups;
    const Side& sd = p.s[which];
    const int h0 = ((int)blockIdx.y - (which ? p.s[0].groups : 0)) * p.per, h1 = min(sd.H, h0 + p.per);
    const long long tok = (long long)blockIdx.x * RPB + threadIdx.x / LPR;
    const bool in = tok < p.tokens;
    const long long token = in ? tok : p.tokens - 1;
    const long long b = token / p.N, n = token % p.N;
    const T* x = static_cast<const T*>(sd.x) + b * sd.xs.b + n * sd.xs.n + l * EPV;
    T* y = static_cast<T*>(sd.y) + (b * sd.H * p.N + n) * D + l * EPV;
    pdl_wait();
    // y = r (x c w + x' s w'), x' and w' the pair's other channel: the weights are
    // taken into the cosines and sines once per token, and a row's lanes exchange
    // x as it was loaded
    TU turn;
    turn.load(p, token, l);
    if (sd.w) {
        const int from = (l + turn.partner - (int)threadIdx.x % 32) * EPV;
        float w[EPV];
#pragma unroll
        for (int e = 0; e < EPV; ++e) w[e] = sd.w[from + (PAIRS ? e ^ 1 : e)];
#pragma unroll
        for (int e = 0; e < EPV; ++e) turn.s[e] *= w[e];
#pragma unroll
        for (int e = 0; e < EPV; ++e) turn.c[e] *= sd.w[l * EPV + e];
    }
    for (int h = h0; h < h1; h += kInFlight) {
        uint4 raw[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u)
            if (h + u < h1) raw[u] = ldg_stream(x + (h + u) * sd.xs.h);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            if (h + u >= h1) break;
            float f[EPV], o[EPV], ss = 0.f;
            Vec16<T>::unpack(raw[u], f);
#pragma unroll
            for (int e = 0; e < EPV; ++e) ss = fmaf(f[e], f[e], ss);
            float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
            if (turn.bad) r = NAN;
            turn.others(raw[u], f, o);
#pragma unroll
            for (int e = 0; e < EPV; ++e) f[e] = r * fmaf(f[e], turn.c[e], o[e] * turn.s[e]);
            if (in) *reinterpret_cast<uint4*>(y + (long long)(h + u) * p.N * D) = Vec16<T>::pack(f);
        }
    }
}

// A CTA runs over tokens blockIdx.x, blockIdx.x + gridDim.x, ... and keeps its
// lanes' part of dw in registers; its sum goes to row blockIdx.y * gridDim.x +
// blockIdx.x of `part`, and qk_rope_weights_kernel adds the rows in order.
template <typename T, int D, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qk_rope_bwd_kernel(const __grid_constant__ Args p) {
    using TU = Turn<T, D, PAIRS>;
    constexpr int EPV = TU::EPV, LPR = TU::LPR, RPB = kThreads / LPR;
    // one row each of x and dy: more only costs registers and with them warps
    // (3x1777x(12+4)x128 fp32: 42 us with two rows, 36 with one; 2x4096x(8+8)x64
    // bf16: 31 and 25)
    constexpr int U = 1;
    __shared__ float red[RPB][D];
    const int l = threadIdx.x % LPR;
    const int which = (int)blockIdx.y >= p.s[0].groups;
    const Side& sd = p.s[which];
    const int h0 = ((int)blockIdx.y - (which ? p.s[0].groups : 0)) * p.per, h1 = min(sd.H, h0 + p.per);
    pdl_wait();
    float w[EPV], dw[EPV] = {};
#pragma unroll
    for (int e = 0; e < EPV; ++e) w[e] = sd.w ? sd.w[l * EPV + e] : 1.f;
    for (long long t0 = (long long)blockIdx.x * RPB; t0 < p.tokens; t0 += (long long)gridDim.x * RPB) {
        const long long tok = t0 + threadIdx.x / LPR;
        const bool in = tok < p.tokens;
        const long long token = in ? tok : p.tokens - 1;
        const long long b = token / p.N, n = token % p.N;
        const T* x = static_cast<const T*>(sd.x) + b * sd.xs.b + n * sd.xs.n + l * EPV;
        const T* dy = static_cast<const T*>(sd.dy) + (b * sd.H * p.N + n) * D + l * EPV;
        T* dx = static_cast<T*>(sd.y) + b * sd.ys.b + n * sd.ys.n + l * EPV;
        TU turn;
        turn.load(p, token, l);
        for (int h = h0; h < h1; h += U) {
            uint4 rx[U], ry[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (h + u < h1) {
                    rx[u] = ldg_stream(x + (h + u) * sd.xs.h);
                    ry[u] = ldg_stream(dy + (long long)(h + u) * p.N * D);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h + u >= h1) break;
                float f[EPV], g[EPV], o[EPV], ss = 0.f, m = 0.f;
                Vec16<T>::unpack(rx[u], f);
                Vec16<T>::unpack(ry[u], g);
#pragma unroll
                for (int e = 0; e < EPV; ++e) ss = fmaf(f[e], f[e], ss);
                float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
                if (turn.bad) r = NAN;
                turn.others(ry[u], g, o);
#pragma unroll
                for (int e = 0; e < EPV; ++e) {  // g: v, R turned back
                    g[e] = fmaf(g[e], turn.c[e], o[e] * -turn.s[e]);
                    f[e] *= r;
                    if (in) dw[e] = fmaf(g[e], f[e], dw[e]);
                    g[e] *= w[e];
                    m = fmaf(g[e], f[e], m);
                }
                m = row_sum<LPR>(m) * (1.f / D);
#pragma unroll
                for (int e = 0; e < EPV; ++e) f[e] = r * (g[e] - f[e] * m);
                if (in) *reinterpret_cast<uint4*>(dx + (h + u) * sd.ys.h) = Vec16<T>::pack(f);
            }
        }
    }
    if (p.part == nullptr) return;
#pragma unroll
    for (int e = 0; e < EPV; ++e) red[threadIdx.x / LPR][l * EPV + e] = dw[e];
    __syncthreads();
    for (int a = threadIdx.x; a < D; a += kThreads) {
        float sum = 0.f;
        for (int r = 0; r < RPB; ++r) sum += red[r][a];
        p.part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * D + a] = sum;
    }
}

// dw: rows of `part` in a fixed order. A block adds 16 columns of the queries'
// rows or of the keys' (64 slices of the rows, then the slices).
constexpr int kColumns = 16, kSlices = 1024 / kColumns;
__global__ void __launch_bounds__(1024)
qk_rope_weights_kernel(const float* __restrict__ part, int rows_q, int rows_k, int d, float* dwq, float* dwk) {
    __shared__ float red[kSlices][kColumns + 1];
    const int c = threadIdx.x % kColumns, s = threadIdx.x / kColumns;
    const bool keys = (int)blockIdx.x >= d / kColumns;
    const int a = (blockIdx.x % (d / kColumns)) * kColumns + c, rows = keys ? rows_k : rows_q;
    const float* src = part + (keys ? (size_t)rows_q * d : 0) + a;
    pdl_wait();
    float sum = 0.f;
#pragma unroll 8
    for (int r = s; r < rows; r += kSlices) sum += src[(size_t)r * d];
    red[s][c] = sum;
    __syncthreads();
    if (threadIdx.x < 32 * kColumns) {  // a warp per column
        const int col = threadIdx.x / 32, l = threadIdx.x % 32;
        float x = red[l][col] + red[l + 32][col];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (l == 0) (keys ? dwk : dwq)[(blockIdx.x % (d / kColumns)) * kColumns + col] = x;
    }
}

int lanes_per_row(const la_rope_desc& p) { return p.dtype == LA_F32 ? p.d / 4 : p.d / 8; }

// Heads per group: as many as leave the GPU full of threads, so that a
// token's cosines and sines are loaded once for them; single heads when
// there are few tokens.
int heads_per_group(const la_rope_desc& p, int sms) {
    const long long lanes = (long long)p.B * p.N * lanes_per_row(p);
    int per = 16;
    while (per > 1 && lanes * ((p.Hq + per - 1) / per + (p.Hk + per - 1) / per) < (long long)sms * 2048) per /= 2;
    return per;
}

struct Grid {
    int per, gq, gk, x;
};
Grid backward_grid(const la_rope_desc& p, int sms) {
    Grid g;
    g.per = heads_per_group(p, sms);
    g.gq = (p.Hq + g.per - 1) / g.per;
    g.gk = (p.Hk + g.per - 1) / g.per;
    const long long rpb = kThreads / lanes_per_row(p), blocks = ((long long)p.B * p.N + rpb - 1) / rpb;
    // as many rounds over the tokens for every CTA, at most 16 CTAs per SM in all
    const long long fill = ((long long)sms * 16 + g.gq + g.gk - 1) / (g.gq + g.gk);
    const long long rounds = (blocks + fill - 1) / fill;
    g.x = (int)((blocks + rounds - 1) / rounds);
    return g;
}

template <typename F> cudaError_t dispatch(const la_rope_desc& p, F f) {
    auto with = [&](auto t, auto d) -> cudaError_t {
        return p.interleaved ? f(t, d, std::true_type{}) : f(t, d, std::false_type{});
    };
    auto with_d = [&](auto t) -> cudaError_t {
        switch (p.d) {
            case 16: return with(t, std::integral_constant<int, 16>{});
            case 32: return with(t, std::integral_constant<int, 32>{});
            case 64: return with(t, std::integral_constant<int, 64>{});
            case 128: return with(t, std::integral_constant<int, 128>{});
        }
        return cudaErrorInvalidValue;
    };
    return p.dtype == LA_F32 ? with_d(float{}) : with_d(__nv_bfloat16{});
}

Args make_args(const la_rope_desc& p, const float* cos, const float* sin, const int32_t* positions, int per) {
    Args a = {};
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    a.tokens = (long long)p.B * p.N;
    a.N = p.N;
    a.rot = p.rot;
    a.rows = p.table_rows;
    a.per = per;
    a.eps = p.eps;
    return a;
}

}  // namespace

size_t qk_rope_partials(const la_rope_desc& p, int sms) {
    const Grid g = backward_grid(p, sms);
    return (size_t)(g.gq + g.gk) * g.x;
}

cudaError_t qk_norm_rope(const la_rope_desc& p, const void* q, const la_strides& qs, const void* k, const la_strides& ks,
                         const float* wq, const float* wk, const float* cos, const float* sin, const int32_t* positions,
                         void* q_out, void* k_out, cudaStream_t st) {
    const int per = heads_per_group(p, device_sms());
    Args a = make_args(p, cos, sin, positions, per);
    a.s[0] = Side{q, nullptr, q_out, wq, qs, qs, p.Hq, (p.Hq + per - 1) / per};
    a.s[1] = Side{k, nullptr, k_out, wk, ks, ks, p.Hk, (p.Hk + per - 1) / per};
    return dispatch(p, [&](auto t, auto d, auto pairs) {
        using T = decltype(t);
        constexpr int D = decltype(d)::value;
        constexpr long long rpb = kForward / (D / Vec16<T>::N);
        const dim3 grid((unsigned)((a.tokens + rpb - 1) / rpb), (unsigned)(a.s[0].groups + a.s[1].groups));
        return launch_pdl(qk_rope_kernel<T, D, decltype(pairs)::value>, grid, dim3(kForward), 0, st, a);
    });
}

cudaError_t qk_norm_rope_backward(const la_rope_desc& p, const void* q, const la_strides& qs, const void* k,
                                  const la_strides& ks, const float* wq, const float* wk, const float* cos,
                                  const float* sin, const int32_t* positions, const void* dq_out, const void* dk_out,
                                  void* dq, const la_strides& dqs, void* dk, const la_strides& dks, float* dwq, float* dwk,
                                  float* part, cudaStream_t st) {
    const Grid g = backward_grid(p, device_sms());
    Args a = make_args(p, cos, sin, positions, g.per);
    a.s[0] = Side{q, dq_out, dq, wq, qs, dqs, p.Hq, g.gq};
    a.s[1] = Side{k, dk_out, dk, wk, ks, dks, p.Hk, g.gk};
    a.part = dwq ? part : nullptr;
    const cudaError_t e = dispatch(p, [&](auto t, auto d, auto pairs) {
        return launch_pdl(qk_rope_bwd_kernel<decltype(t), decltype(d)::value, decltype(pairs)::value>,
                          dim3((unsigned)g.x, (unsigned)(g.gq + g.gk)), dim3(kThreads), 0, st, a);
    });
    if (e != cudaSuccess || dwq == nullptr) return e;
    return launch_pdl(qk_rope_weights_kernel, dim3(2 * (unsigned)p.d / kColumns), dim3(1024), 0, st, static_cast<const float*>(part), g.gq * g.x,
                      g.gk * g.x, p.d, dwq, dwk);
}

}  // namespace la
