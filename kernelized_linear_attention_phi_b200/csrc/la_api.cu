// C ABI of libla_b200 (declared in include/la.h): argument validation,
// workspace planning and kernel dispatch. Validation is fail-closed: a bad
// request returns a status before anything is launched.

#include <la.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "common.cuh"
#include "device.h"
#include "gated.h"
#include "internal.h"
#include "launch_util.h"
#include "plan.h"
#include "qk_rope.h"
#include "tc.h"
#include "tc_common.cuh"

namespace la {
namespace {

constexpr int kSimtChunk = 64;     // chunk length the SIMT chunked kernel runs at
constexpr size_t kAlign = 256;
constexpr int kGatedRow = 1 << 30;  // tokens of a gated row: its kernels' row numbers stay below 2^31

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

la_status check_desc(const la_desc* d) {
    if (d == nullptr) return LA_ERR_INVALID_ARG;
    if (d->B <= 0 || d->H <= 0 || d->N <= 0 || d->d <= 0) return LA_ERR_INVALID_ARG;
    if (d->dtype != LA_F32 && d->dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (d->phi != LA_PHI_RELU1 && d->phi != LA_PHI_IDENTITY && d->phi != LA_PHI_ELU1) return LA_ERR_INVALID_ARG;
    if (d->normalize != 0 && d->normalize != 1) return LA_ERR_INVALID_ARG;
    if (d->d != 16 && d->d != 32 && d->d != 64 && d->d != 128) return LA_ERR_UNSUPPORTED;
    if (d->normalize == 1 && d->phi == LA_PHI_IDENTITY) return LA_ERR_UNSUPPORTED;
    if ((long long)d->B * d->H > 65535) return LA_ERR_UNSUPPORTED;  // grid.y limit
    if ((long long)d->B * d->H * d->N * d->d > (1LL << 40)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

la_status check_chunk(int chunk) { return (chunk == 64 || chunk == 128) ? LA_OK : LA_ERR_UNSUPPORTED; }

// The library's kernels are built for sm_100a only.
la_status check_device() {
    static std::atomic<uint64_t> ok{0}, bad{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return LA_ERR_CUDA;
    }
    const uint64_t bit = 1ull << (dev & 63);
    if (ok.load() & bit) return LA_OK;
    if (bad.load() & bit) return LA_ERR_UNSUPPORTED;
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) {
        cudaGetLastError();
        return LA_ERR_CUDA;
    }
    if (major != 10) {
        bad.fetch_or(bit);
        return LA_ERR_UNSUPPORTED;
    }
    ok.fetch_or(bit);
    return LA_OK;
}

Problem to_problem(const la_desc* d) {
    return Problem{d->B, d->H, d->N, d->d, d->dtype, d->phi, d->normalize};
}

// ---- work plans (pure functions of the problem, shared by sizing and launch) ----

// Plans for the current device's SM count (plan.h): a workspace sized on a
// device fits every launch on that device.
plan::SplitPlan kv_plan(const Problem& p) { return plan::kv_plan(p, device_sms()); }
plan::BlockPlan block_plan(const Problem& p) { return plan::block_plan(p, device_sms()); }
using plan::BlockPlan;
using plan::SplitPlan;
BlockPlan gated_plan(const Problem& p, bool backward) {
    return plan::gated_plan(p, device_sms(), plan::gated_ctas_per_sm(p, backward), backward);
}

int prefix_nbins(const Problem& p, int kchunk) { return p.N / kchunk + 1; }

struct WsLayout {
    size_t part = 0, sz = 0, perm = 0, msort = 0, bins = 0, total = 0;
    size_t grec = 0, gtot = 0, gn = 0, gden = 0;  // gradients
    size_t dec = 0, gates = 0, up = 0, col = 0, own = 0, dgp = 0, chunks = 0;  // gated forms
};

WsLayout ws_layout(const Problem& p, int op) {
    WsLayout L;
    size_t off = WS_HEADER;
    const size_t rec = p.state_floats() * sizeof(float);
    if (op == LA_OP_KV_SUMMARY || op == LA_OP_NONCAUSAL) {
        size_t nrec;
        if (tc_supported(p)) {
            const KvBalanced w = kv_balanced_plan(p);
            nrec = (size_t)w.G * w.K;
        } else {
            nrec = (size_t)p.bh() * kv_plan(p).nsplit;
        }
        L.part = off;
        off = round_up(off + nrec * rec, kAlign);
        if (op == LA_OP_NONCAUSAL) {
            L.sz = off;
            off = round_up(off + (size_t)p.bh() * rec, kAlign);
        }
    } else if (op == LA_OP_CAUSAL || op == LA_OP_PREFIX) {
        const BlockPlan bp = block_plan(p);
        L.part = off;
        off = round_up(off + (size_t)p.bh() * bp.nblk * rec, kAlign);
        if (op == LA_OP_PREFIX) {
            const int nbins = prefix_nbins(p, 64);  // the most bins any kernel uses
            L.perm = off;
            off = round_up(off + sizeof(int32_t) * (size_t)p.B * p.N, kAlign);
            L.msort = off;
            off = round_up(off + sizeof(int32_t) * (size_t)p.B * p.N, kAlign);
            L.bins = off;
            off = round_up(off + sizeof(int32_t) * (size_t)p.B * (nbins + 1), kAlign);
        }
    } else if (op == LA_OP_NONCAUSAL_BWD || op == LA_OP_CAUSAL_BWD) {
        const BlockPlan bp = block_plan(p);
        L.part = off;
        if (op == LA_OP_NONCAUSAL_BWD) {
            // the KV summary's own scratch where kv_summary_impl expects it
            // (on the tensor cores it then takes the gradient kernels' (G, h)
            // records, whose split may have more slots), then the totals
            // (S, z) and (G, h)
            off = ws_layout(p, LA_OP_KV_SUMMARY).total;
            if (tc_supported(p)) off = std::max(off, round_up(L.part + tc_backward_record_slots(p) * rec, kAlign));
            L.sz = off;
            off = round_up(off + (size_t)p.bh() * rec, kAlign);
            L.gtot = off;
            off = round_up(off + (size_t)p.bh() * rec, kAlign);
            if (tc_supported(p)) {  // the CUDA-core path's block states and gn, gden are not used
                L.total = off;
                return L;
            }
        } else {
            off = round_up(off + (size_t)p.bh() * bp.nblk * rec, kAlign);  // block states (S, z)
        }
        L.grec = off;
        off = round_up(off + (size_t)p.bh() * bp.nblk * rec, kAlign);      // block states (G, h)
        L.gn = off;
        off = round_up(off + sizeof(float) * (size_t)p.bh() * p.N * p.d, kAlign);
        L.gden = off;
        off = round_up(off + sizeof(float) * (size_t)p.bh() * p.N, kAlign);
    } else if (op == LA_OP_GATED_CAUSAL || op == LA_OP_GATED_CAUSAL_BWD) {
        if (p.N > kGatedRow) return L;
        const bool bwd = op == LA_OP_GATED_CAUSAL_BWD;
        const BlockPlan bp = gated_plan(p, bwd);
        const bool tcf = !bwd && tc_gated_supported(p);  // forms the last state from a record too
        if (bp.nblk > 1 || tcf) {  // block states and the products of the blocks' gates
            L.part = off;
            off = round_up(off + (size_t)p.bh() * bp.nblk * rec, kAlign);
            L.dec = off;
            off = round_up(off + (size_t)p.bh() * bp.nblk * sizeof(float), kAlign);
        }
        if (!tcf) {
            L.gates = off;
            off = round_up(off + gated_gate_bytes(p), kAlign);
        }
        if (bwd) {
            const size_t tokens = (size_t)p.bh() * p.N * sizeof(float);
            L.up = off;
            off = round_up(off + tokens, kAlign);
            L.col = off;
            off = round_up(off + tokens, kAlign);
            L.own = off;
            off = round_up(off + tokens, kAlign);
            L.dgp = off;
            off = round_up(off + tokens, kAlign);
            L.chunks = off;
            off = round_up(off + (size_t)p.bh() * cdiv(p.N, gated_chunk(p)) * gated_chunk_state_bytes(p), kAlign);
        }
    } else {
        return L;
    }
    L.total = off;
    return L;
}

template <typename P>
P* at(void* ws, size_t off) {
    return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

la_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return LA_OK;
    cudaGetLastError();
    return LA_ERR_CUDA;
}

la_status check_ws(const WsLayout& L, void* ws, size_t ws_bytes) {
    if (ws == nullptr || ws_bytes < L.total) return LA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LA_ERR_MISALIGNED;
    return LA_OK;
}

#define LA_TRY(expr)                      \
    do {                                  \
        la_status s__ = (expr);           \
        if (s__ != LA_OK) return s__;     \
    } while (0)

la_status check_rope(const la_rope_desc* d) {
    if (d == nullptr) return LA_ERR_INVALID_ARG;
    if (d->B <= 0 || d->N <= 0 || d->Hq <= 0 || d->Hk <= 0 || d->d <= 0) return LA_ERR_INVALID_ARG;
    if (d->dtype != LA_F32 && d->dtype != LA_BF16) return LA_ERR_INVALID_ARG;
    if (d->interleaved != 0 && d->interleaved != 1) return LA_ERR_INVALID_ARG;
    if (d->rot < 0 || d->table_rows < 0 || !(d->eps >= 0.f) || !std::isfinite(d->eps)) return LA_ERR_INVALID_ARG;
    if (d->d != 16 && d->d != 32 && d->d != 64 && d->d != 128) return LA_ERR_UNSUPPORTED;
    if (d->rot > d->d || d->rot % 16 != 0) return LA_ERR_UNSUPPORTED;
    if (d->rot > 0 && d->table_rows == 0) return LA_ERR_INVALID_ARG;
    if (d->Hq > 32767 || d->Hk > 32767) return LA_ERR_UNSUPPORTED;  // grid.y limit
    if ((long long)d->B * d->N >= (1LL << 31)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Whether two rows of a [B, N, H, d] view share an element (strides >= d).
bool rows_overlap(const la_rope_desc& d, const la_strides& s, int H) {
    struct Dim {
        long long size, stride;
    } dim[3] = {{d.B, s.b}, {d.N, s.n}, {H, s.h}};
    for (Dim& x : dim)
        if (x.size == 1) x.stride = 0;
    std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    __int128 extent = d.d;  // the usual views nest: each stride steps over all that lies below it
    bool nested = true;
    for (const Dim& x : dim) {
        if (x.size == 1) continue;
        nested = nested && x.stride >= extent;
        extent += (__int128)x.stride * (x.size - 1);
    }
    if (nested) return false;
    // others: a difference of indexes, not all 0, that moves by less than a row;
    // the longest dimension's part follows from those of the other two
    std::sort(dim, dim + 3, [](const Dim& a, const Dim& b) { return a.size < b.size; });
    const Dim &x = dim[0], &y = dim[1], &z = dim[2];
    for (long long i = 0; i < x.size; ++i)
        for (long long j = i ? 1 - y.size : 0; j < y.size; ++j) {
            const __int128 at = (__int128)i * x.stride + (__int128)j * y.stride;
            const __int128 mag = at < 0 ? -at : at;
            // k * stride next to mag on either side (the sign of k is free); k = 0 alone
            // is no difference of rows
            const __int128 k = mag / z.stride, low = mag - k * z.stride;
            if (k < z.size && low < d.d && (i || j || k)) return true;
            if (k + 1 < z.size && z.stride - low < d.d) return true;
        }
    return false;
}

// A [B, N, H, d] view: strides in multiples of 16 bytes, not negative; rows of
// an output must not fall on one another.
la_status check_strides(const la_rope_desc& d, const la_strides& s, int H, bool output) {
    const long long unit = d.dtype == LA_F32 ? 4 : 8;
    const long long size[3] = {d.B, d.N, H}, stride[3] = {s.b, s.n, s.h};
    for (int i = 0; i < 3; ++i) {
        if (size[i] == 1) continue;
        if (stride[i] < 0 || (output && stride[i] < d.d)) return LA_ERR_INVALID_ARG;
        if (stride[i] % unit != 0) return LA_ERR_MISALIGNED;
    }
    return output && rows_overlap(d, s, H) ? LA_ERR_INVALID_ARG : LA_OK;
}

la_status check_rope_inputs(const la_rope_desc& d, const void* q, const la_strides* qs, const void* k,
                            const la_strides* ks, const float* wq, const float* wk, const float* cos, const float* sin,
                            const int32_t* positions) {
    if (!q || !k || !qs || !ks) return LA_ERR_INVALID_ARG;
    if ((wq == nullptr) != (wk == nullptr)) return LA_ERR_INVALID_ARG;
    if (d.rot > 0 && (!cos || !sin)) return LA_ERR_INVALID_ARG;
    if (d.rot > 0 && !positions && d.table_rows < d.N) return LA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, static_cast<const void*>(wq), static_cast<const void*>(wk),
                            static_cast<const void*>(cos), static_cast<const void*>(sin),
                            static_cast<const void*>(positions)})
        if (!aligned16(ptr)) return LA_ERR_MISALIGNED;
    LA_TRY(check_strides(d, *qs, d.Hq, false));
    return check_strides(d, *ks, d.Hk, false);
}

la_status kv_summary_impl(const Problem& p, const void* k, const void* v, float* S, float* z,
                          void* ws, cudaStream_t st) {
    float* part = at<float>(ws, ws_layout(p, LA_OP_KV_SUMMARY).part);
    if (tc_noncausal_fused_supported(p))  // small problems: one launch, reduced in a cluster per head
        return cuda_status(tc_noncausal_fused(p, nullptr, k, v, nullptr, S, z, at<uint32_t>(ws, 0), st));
    if (tc_supported(p)) return cuda_status(tc_kv_summary(p, k, v, part, S, z, at<uint32_t>(ws, 0), st));
    const SplitPlan sp = kv_plan(p);
    if (tc_f32_supported(p)) {
        LA_TRY(cuda_status(tc_f32_states(p, k, v, sp.tps, sp.nsplit, part, at<uint32_t>(ws, 0), st)));
    } else {
        LA_TRY(cuda_status(simt_kv_partial(p, k, v, sp.tps, sp.nsplit, part, st)));
    }
    return cuda_status(state_reduce(p, part, sp.nsplit, S, z, st));
}

}  // namespace

la_status kv_summary_args(const la_desc* desc, const void* k, const void* v, const float* S_out,
                          const float* z_out) {
    LA_TRY(check_desc(desc));
    if (!k || !v || !S_out || !z_out) return LA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(S_out) || !aligned16(z_out)) return LA_ERR_MISALIGNED;
    return LA_OK;
}

la_status kv_summary_checked(const la_desc* desc, const void* k, const void* v, float* S_out,
                             float* z_out, void* ws, size_t ws_bytes, cudaStream_t st) {
    LA_TRY(kv_summary_args(desc, k, v, S_out, z_out));
    const Problem p = to_problem(desc);
    LA_TRY(check_ws(ws_layout(p, LA_OP_KV_SUMMARY), ws, ws_bytes));
    LA_TRY(check_device());
    timing_begin(st);
    return kv_summary_impl(p, k, v, S_out, z_out, ws, st);
}

}  // namespace la

using namespace la;

extern "C" {

int32_t la_version(void) { return 100; }

const char* la_status_string(la_status s) {
    switch (s) {
        case LA_OK: return "LA_OK";
        case LA_ERR_INVALID_ARG: return "LA_ERR_INVALID_ARG";
        case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED";
        case LA_ERR_MISALIGNED: return "LA_ERR_MISALIGNED";
        case LA_ERR_WORKSPACE: return "LA_ERR_WORKSPACE";
        case LA_ERR_CUDA: return "LA_ERR_CUDA";
        case LA_ERR_MASK_RANGE: return "LA_ERR_MASK_RANGE";
        case LA_ERR_TIMEOUT: return "LA_ERR_TIMEOUT";
    }
    return "LA_ERR_UNKNOWN";
}

size_t la_workspace_size(const la_desc* desc, int32_t op, int32_t chunk) {
    if (check_desc(desc) != LA_OK) return 0;
    if ((op == LA_OP_CAUSAL || op == LA_OP_PREFIX) && check_chunk(chunk) != LA_OK) return 0;
    if (op < LA_OP_KV_SUMMARY || op > LA_OP_GATED_CAUSAL_BWD) return 0;
    return ws_layout(to_problem(desc), op).total;
}

la_status la_kv_summary(const la_desc* desc, const void* k, const void* v, float* S_out,
                        float* z_out, void* ws, size_t ws_bytes, void* stream) {
    return la::kv_summary_checked(desc, k, v, S_out, z_out, ws, ws_bytes,
                                  static_cast<cudaStream_t>(stream));
}

la_status la_noncausal(const la_desc* desc, const void* q, const void* k, const void* v, void* out,
                       float* S_out, float* z_out, void* ws, size_t ws_bytes, void* stream) {
    LA_TRY(check_desc(desc));
    if (!q || !k || !v || !out) return LA_ERR_INVALID_ARG;
    if ((S_out == nullptr) != (z_out == nullptr)) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return LA_ERR_MISALIGNED;
    if (S_out && (!aligned16(S_out) || !aligned16(z_out))) return LA_ERR_MISALIGNED;
    const Problem p = to_problem(desc);
    const WsLayout L = ws_layout(p, LA_OP_NONCAUSAL);
    LA_TRY(check_ws(L, ws, ws_bytes));
    LA_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    timing_begin(st);
    // small problems: one kernel, a thread-block cluster per head (bf16,
    // d = 64) or one CTA per head (d <= 32)
    if (simt_noncausal_small_supported(p))
        return cuda_status(simt_noncausal_small(p, q, k, v, out, S_out, z_out, st));
    if (tc_noncausal_fused_supported(p))
        return cuda_status(tc_noncausal_fused(p, q, k, v, out, S_out, z_out, at<uint32_t>(ws, 0), st));
    float* S = S_out;
    float* z = z_out;
    if (S == nullptr) {
        S = at<float>(ws, L.sz);
        z = S + (size_t)p.bh() * p.d * p.d;
    }
    LA_TRY(kv_summary_impl(p, k, v, S, z, ws, st));
    if (tc_supported(p)) return cuda_status(tc_readout(p, q, S, z, out, at<uint32_t>(ws, 0), st));
    if (tc_f32_supported(p)) {
        const BlockPlan bp = block_plan(p);
        return cuda_status(tc_f32_readout(p, q, S, z, bp.block_tokens, bp.nblk, out, at<uint32_t>(ws, 0), st));
    }
    return cuda_status(simt_readout(p, q, S, z, out, st));
}

}  // extern "C"

namespace la {
namespace {

// Causal outputs; with S_total/z_total (both or neither) also the state after
// the last token, written by the block-state scan.
la_status causal_impl(const la_desc* desc, int32_t chunk, const void* q, const void* k, const void* v,
                      void* out, float* S_total, float* z_total, void* ws, size_t ws_bytes,
                      cudaStream_t st) {
    LA_TRY(check_desc(desc));
    LA_TRY(check_chunk(chunk));
    if (!q || !k || !v || !out) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return LA_ERR_MISALIGNED;
    if (S_total && (!aligned16(S_total) || !aligned16(z_total))) return LA_ERR_MISALIGNED;
    const Problem p = to_problem(desc);
    const WsLayout L = ws_layout(p, LA_OP_CAUSAL);
    LA_TRY(check_ws(L, ws, ws_bytes));
    LA_TRY(check_device());
    timing_begin(st);
    const BlockPlan bp = block_plan(p);
    float* part = at<float>(ws, L.part);
    // phase 1: per-block states; phase 2: exclusive prefix over blocks (and
    // the total); phase 3: each block's outputs from its prefix state.
    uint32_t* flags = at<uint32_t>(ws, 0);
    if (tc_supported(p) && p.d == 128 && S_total == nullptr && bp.nblk >= 2) {
        // the states of every block but the last (no block's prefix holds
        // it), then the sweep, whose CTAs each sum the states before their
        // block: no scan kernel in between
        LA_TRY(cuda_status(tc_kv_blocks(p, k, v, bp.block_tokens, bp.nblk, part, flags, st, bp.nblk - 1)));
        return cuda_status(tc_chunked_t(p, q, k, v, part, bp.block_tokens, bp.nblk, nullptr, nullptr, nullptr, 0,
                                        out, flags, st, true));
    }
    if (tc_kv_scan_supported(p, bp.block_tokens, bp.nblk)) {  // phases 1 and 2 in one kernel
        LA_TRY(cuda_status(tc_kv_blocks_scan(p, k, v, bp.block_tokens, bp.nblk, part, S_total, z_total, flags, st)));
    } else {
        if (tc_supported(p)) {
            LA_TRY(cuda_status(tc_kv_blocks(p, k, v, bp.block_tokens, bp.nblk, part, flags, st)));
        } else if (tc_f32_supported(p)) {
            LA_TRY(cuda_status(tc_f32_states(p, k, v, bp.block_tokens, bp.nblk, part, flags, st)));
        } else {
            LA_TRY(cuda_status(simt_kv_partial(p, k, v, bp.block_tokens, bp.nblk, part, st)));
        }
        LA_TRY(cuda_status(state_exclusive_scan(p, part, bp.nblk, S_total, z_total, st)));
    }
    if (tc_supported(p))
        return cuda_status(tc_chunked(p, chunk, q, k, v, part, bp.block_tokens, bp.nblk, nullptr,
                                      nullptr, nullptr, 0, out, flags, st));
    if (tc_f32_supported(p))
        return cuda_status(tc_f32_chunked(p, q, k, v, part, bp.block_tokens, bp.nblk, out, flags, st));
    return cuda_status(simt_chunked(p, q, k, v, part, bp.block_tokens, bp.nblk, nullptr, nullptr,
                                    nullptr, 0, out, st));
}

// Gradients of the non-causal or causal form (see la.h): states of the
// forward, a forward sweep for dq, gn, gden and per-block (G, h), the
// suffix (causal) or total (non-causal) of (G, h), a reverse sweep for dk, dv.
la_status backward_impl(const la_desc* desc, bool causal, const void* q, const void* k, const void* v,
                        const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                        cudaStream_t st) {
    LA_TRY(check_desc(desc));
    if (!q || !k || !v || !dout || !dq || !dk || !dv) return LA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, v, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                            static_cast<const void*>(dv)})
        if (!aligned16(ptr)) return LA_ERR_MISALIGNED;
    const Problem p = to_problem(desc);
    const WsLayout L = ws_layout(p, causal ? LA_OP_CAUSAL_BWD : LA_OP_NONCAUSAL_BWD);
    LA_TRY(check_ws(L, ws, ws_bytes));
    LA_TRY(check_device());
    timing_begin(st);
    const BlockPlan bp = block_plan(p);
    if (bp.block_tokens % bwd_chunk(p) != 0) return LA_ERR_UNSUPPORTED;
    const long long rec = (long long)p.state_floats();
    float* grec = at<float>(ws, L.grec);
    float* gn = at<float>(ws, L.gn);
    float* gden = at<float>(ws, L.gden);
    if (causal) {
        float* part = at<float>(ws, L.part);
        uint32_t* flags = at<uint32_t>(ws, 0);
        if (tc_kv_scan_supported(p, bp.block_tokens, bp.nblk)) {
            LA_TRY(cuda_status(tc_kv_blocks_scan(p, k, v, bp.block_tokens, bp.nblk, part, nullptr, nullptr, flags, st)));
        } else {
            if (tc_supported(p)) {
                LA_TRY(cuda_status(tc_kv_blocks(p, k, v, bp.block_tokens, bp.nblk, part, flags, st)));
            } else if (tc_f32_supported(p)) {
                LA_TRY(cuda_status(tc_f32_states(p, k, v, bp.block_tokens, bp.nblk, part, flags, st)));
            } else {
                LA_TRY(cuda_status(simt_kv_partial(p, k, v, bp.block_tokens, bp.nblk, part, st)));
            }
            LA_TRY(cuda_status(state_exclusive_scan(p, part, bp.nblk, nullptr, nullptr, st)));
        }
        const bool tcq = tc_causal_backward_supported(p, bp.block_tokens);
        if (tcq) {  // tensor cores; gn in bf16
            LA_TRY(cuda_status(tc_causal_backward_q(p, q, k, v, dout, part, bp.block_tokens, bp.nblk, dq, gn, gden,
                                                    grec, flags, st)));
        } else {
            LA_TRY(cuda_status(bwd_q(p, true, q, k, v, dout, part, part + (size_t)p.d * p.d, rec, rec,
                                     bp.block_tokens, bp.nblk, dq, gn, gden, grec, st)));
        }
        LA_TRY(cuda_status(state_exclusive_scan(p, grec, bp.nblk, nullptr, nullptr, st, true)));
        if (tcq)
            return cuda_status(tc_causal_backward_kv(p, q, k, v, gn, gden, grec, bp.block_tokens, bp.nblk, dk, dv,
                                                     flags, st));
        return cuda_status(bwd_kv(p, true, q, k, v, gn, gden, grec, grec + (size_t)p.d * p.d, rec, rec,
                                  bp.block_tokens, bp.nblk, dk, dv, st));
    }
    float* S = at<float>(ws, L.sz);
    float* z = S + (size_t)p.bh() * p.d * p.d;
    float* G = at<float>(ws, L.gtot);
    float* h = G + (size_t)p.bh() * p.d * p.d;
    LA_TRY(kv_summary_impl(p, k, v, S, z, ws, st));
    if (tc_supported(p))  // tensor cores: the KV summary's record slots take the (G, h) records
        return cuda_status(tc_noncausal_backward(p, q, k, v, dout, S, z, at<float>(ws, L.part), G, h, dq, dk, dv,
                                                 at<uint32_t>(ws, 0), st));
    LA_TRY(cuda_status(bwd_q(p, false, q, k, v, dout, S, z, (long long)p.d * p.d, p.d, bp.block_tokens,
                             bp.nblk, dq, gn, gden, grec, st)));
    LA_TRY(cuda_status(state_reduce(p, grec, bp.nblk, G, h, st)));
    return cuda_status(bwd_kv(p, false, q, k, v, gn, gden, G, h, (long long)p.d * p.d, p.d, bp.block_tokens,
                              bp.nblk, dk, dv, st));
}

}  // namespace
}  // namespace la

extern "C" {

la_status la_noncausal_backward(const la_desc* desc, const void* q, const void* k, const void* v,
                                const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                void* stream) {
    return backward_impl(desc, false, q, k, v, dout, dq, dk, dv, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

la_status la_causal_backward(const la_desc* desc, const void* q, const void* k, const void* v,
                             const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                             void* stream) {
    return backward_impl(desc, true, q, k, v, dout, dq, dk, dv, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

la_status la_causal_chunked(const la_desc* desc, int32_t chunk, const void* q, const void* k,
                            const void* v, void* out, void* ws, size_t ws_bytes, void* stream) {
    return causal_impl(desc, chunk, q, k, v, out, nullptr, nullptr, ws, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

la_status la_causal_prefill(const la_desc* desc, int32_t chunk, const void* q, const void* k,
                            const void* v, void* out, float* S_out, float* z_out, void* ws,
                            size_t ws_bytes, void* stream) {
    if (S_out == nullptr || z_out == nullptr) return LA_ERR_INVALID_ARG;
    return causal_impl(desc, chunk, q, k, v, out, S_out, z_out, ws, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

la_status la_prefix_mask(const la_desc* desc, int32_t chunk, const void* q, const void* k,
                         const void* v, const int32_t* m, void* out, void* ws, size_t ws_bytes,
                         void* stream) {
    LA_TRY(check_desc(desc));
    LA_TRY(check_chunk(chunk));
    if (!q || !k || !v || !m || !out) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(m))
        return LA_ERR_MISALIGNED;
    const Problem p = to_problem(desc);
    if (p.N > (1 << 21)) return LA_ERR_UNSUPPORTED;  // bin table must fit in shared memory
    const WsLayout L = ws_layout(p, LA_OP_PREFIX);
    LA_TRY(check_ws(L, ws, ws_bytes));
    LA_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    timing_begin(st);
    const BlockPlan bp = block_plan(p);
    const bool tc = tc_supported(p);
    const int kchunk = tc ? tc_chunk(p, chunk) : kSimtChunk;  // chunk length of the kernel used
    const int nbins = prefix_nbins(p, kchunk);
    uint32_t* flags = at<uint32_t>(ws, 0);
    int32_t* perm = at<int32_t>(ws, L.perm);
    int32_t* msort = at<int32_t>(ws, L.msort);
    int32_t* bins = at<int32_t>(ws, L.bins);
    float* part = at<float>(ws, L.part);
    // the binning reads only m: launched after the KV pass it runs beside it
    // (bin_kernel waits for its predecessor only at its end); the next
    // kernel (the scan, or the sweep when the KV pass scans in-cluster)
    // waits for both
    const bool cscan = tc_kv_scan_supported(p, bp.block_tokens, bp.nblk);
    if (cscan) {
        LA_TRY(cuda_status(tc_kv_blocks_scan(p, k, v, bp.block_tokens, bp.nblk, part, nullptr, nullptr, flags, st)));
    } else if (tc) {
        LA_TRY(cuda_status(tc_kv_blocks(p, k, v, bp.block_tokens, bp.nblk, part, flags, st)));
    } else if (tc_f32_supported(p)) {
        LA_TRY(cuda_status(tc_f32_states(p, k, v, bp.block_tokens, bp.nblk, part, flags, st)));
    } else {
        LA_TRY(cuda_status(simt_kv_partial(p, k, v, bp.block_tokens, bp.nblk, part, st)));
    }
    LA_TRY(cuda_status(bin_queries(p, m, kchunk, nbins, perm, bins, msort, flags, st)));
    if (!cscan) LA_TRY(cuda_status(state_exclusive_scan(p, part, bp.nblk, nullptr, nullptr, st)));
    if (tc)
        return cuda_status(tc_chunked(p, chunk, q, k, v, part, bp.block_tokens, bp.nblk, perm, bins,
                                      msort, nbins, out, flags, st));
    if (tc_f32_supported(p))  // 64-token chunks, like the CUDA-core kernel
        return cuda_status(tc_f32_prefix(p, q, k, v, part, bp.block_tokens, bp.nblk, perm, bins, msort, nbins, out,
                                         flags, st));
    return cuda_status(simt_chunked(p, q, k, v, part, bp.block_tokens, bp.nblk, perm, bins, msort,
                                    nbins, out, st));
}

la_status la_decode_step(const la_desc* desc, const void* q, const void* k, const void* v, float* S,
                         float* z, void* out, void* stream) {
    if (desc == nullptr) return LA_ERR_INVALID_ARG;
    la_desc d1 = *desc;
    d1.N = 1;  // N is not used by a decode step
    LA_TRY(check_desc(&d1));
    if (!q || !k || !v || !S || !z || !out) return LA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(S) || !aligned16(z) ||
        !aligned16(out))
        return LA_ERR_MISALIGNED;
    LA_TRY(check_device());
    timing_begin(static_cast<cudaStream_t>(stream));
    return cuda_status(decode_step(to_problem(&d1), q, k, v, S, z, out,
                                   static_cast<cudaStream_t>(stream)));
}

la_status la_gated_causal(const la_desc* desc, const void* q, const void* k, const void* v, const void* g,
                          const float* S_in, const float* z_in, void* out, float* S_out, float* z_out, void* ws,
                          size_t ws_bytes, void* stream) {
    LA_TRY(check_desc(desc));
    if (!q || !k || !v || !g || !out) return LA_ERR_INVALID_ARG;
    if ((S_in == nullptr) != (z_in == nullptr) || (S_out == nullptr) != (z_out == nullptr)) return LA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, v, g, static_cast<const void*>(out), static_cast<const void*>(S_in),
                            static_cast<const void*>(z_in), static_cast<const void*>(S_out),
                            static_cast<const void*>(z_out)})
        if (!aligned16(ptr)) return LA_ERR_MISALIGNED;
    const Problem p = to_problem(desc);
    if (p.N > kGatedRow) return LA_ERR_UNSUPPORTED;
    const WsLayout L = ws_layout(p, LA_OP_GATED_CAUSAL);
    LA_TRY(check_ws(L, ws, ws_bytes));
    LA_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    timing_begin(st);
    const BlockPlan bp = gated_plan(p, false);
    // own states of the blocks (the last block's only for the state after it),
    // then the state in front of each, then the outputs
    float* part = at<float>(ws, L.part);
    float* dec = at<float>(ws, L.dec);
    if (tc_gated_supported(p)) {
        uint32_t* flags = at<uint32_t>(ws, 0);
        const int count = S_out ? bp.nblk : bp.nblk - 1;
        if (count == 0)
            return cuda_status(tc_gated_sweep(p, q, k, v, g, nullptr, S_in, z_in, bp.block_tokens, 1, out, flags, st));
        LA_TRY(cuda_status(tc_gated_states(p, false, k, v, g, nullptr, nullptr, bp.block_tokens, bp.nblk, 0, count,
                                           S_out != nullptr, part, dec, flags, st)));
        LA_TRY(cuda_status(gated_scan(p, false, part, dec, bp.nblk, S_in, z_in, S_out, z_out, st)));
        return cuda_status(tc_gated_sweep(p, q, k, v, g, part, nullptr, nullptr, bp.block_tokens, bp.nblk, out, flags, st));
    }
    uint8_t* gates = at<uint8_t>(ws, L.gates);
    LA_TRY(cuda_status(gated_gates(p, g, gates, st)));
    if (bp.nblk == 1)
        return cuda_status(gated_sweep(p, q, k, v, gates, nullptr, S_in, z_in, bp.block_tokens, 1, out, S_out, z_out, st));
    LA_TRY(cuda_status(gated_states(p, false, k, v, gates, nullptr, nullptr, bp.block_tokens, bp.nblk, 0,
                                    S_out ? bp.nblk : bp.nblk - 1, S_out != nullptr, part, dec, st)));
    LA_TRY(cuda_status(gated_scan(p, false, part, dec, bp.nblk, S_in, z_in, S_out, z_out, st)));
    return cuda_status(gated_sweep(p, q, k, v, gates, part, nullptr, nullptr, bp.block_tokens, bp.nblk, out, nullptr,
                                   nullptr, st));
}

la_status la_gated_causal_backward(const la_desc* desc, const void* q, const void* k, const void* v, const void* g,
                                   const void* dout, void* dq, void* dk, void* dv, void* dg, void* ws, size_t ws_bytes,
                                   void* stream) {
    LA_TRY(check_desc(desc));
    if (!q || !k || !v || !g || !dout || !dq || !dk || !dv || !dg) return LA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, v, g, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                            static_cast<const void*>(dv), static_cast<const void*>(dg)})
        if (!aligned16(ptr)) return LA_ERR_MISALIGNED;
    const Problem p = to_problem(desc);
    if (p.N > kGatedRow) return LA_ERR_UNSUPPORTED;
    const WsLayout L = ws_layout(p, LA_OP_GATED_CAUSAL_BWD);
    LA_TRY(check_ws(L, ws, ws_bytes));
    LA_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    timing_begin(st);
    const BlockPlan bp = gated_plan(p, true);
    uint8_t* gates = at<uint8_t>(ws, L.gates);
    LA_TRY(cuda_status(gated_gates(p, g, gates, st)));
    float* up = p.normalize ? at<float>(ws, L.up) : nullptr;
    float* col = p.normalize ? at<float>(ws, L.col) : nullptr;
    float* own = p.normalize ? at<float>(ws, L.own) : nullptr;
    float* dgp = at<float>(ws, L.dgp);
    void* chunks = at<char>(ws, L.chunks);
    float *part = nullptr, *dec = nullptr;
    // block states on the tensor cores where the blocks are long enough to fill
    // their pipeline (4x16x8192x128: 141 -> 70 us in order, 160 -> 82 in reverse)
    const bool tcs = tc_gated_supported(p) && bp.block_tokens >= 256;
    uint32_t* flags = at<uint32_t>(ws, 0);
    if (bp.nblk > 1) {
        part = at<float>(ws, L.part);
        dec = at<float>(ws, L.dec);
        if (tcs)
            LA_TRY(cuda_status(tc_gated_states(p, false, k, v, g, nullptr, nullptr, bp.block_tokens, bp.nblk, 0, bp.nblk - 1,
                                               false, part, dec, flags, st)));
        else
            LA_TRY(cuda_status(gated_states(p, false, k, v, gates, nullptr, nullptr, bp.block_tokens, bp.nblk, 0,
                                        bp.nblk - 1, false, part, dec, st)));
        LA_TRY(cuda_status(gated_scan(p, false, part, dec, bp.nblk, nullptr, nullptr, nullptr, nullptr, st)));
    }
    LA_TRY(cuda_status(gated_bwd_q(p, q, k, v, gates, dout, part, bp.block_tokens, bp.nblk, dq, up, col, own, dgp, chunks,
                                   st)));
    if (bp.nblk > 1) {  // the same records, from the other end
        if (tcs)
            LA_TRY(cuda_status(tc_gated_states(p, true, q, dout, g, up, col, bp.block_tokens, bp.nblk, 1, bp.nblk - 1, false,
                                               part, dec, flags, st)));
        else
            LA_TRY(cuda_status(gated_states(p, true, q, dout, gates, up, col, bp.block_tokens, bp.nblk, 1, bp.nblk - 1, false,
                                        part, dec, st)));
        LA_TRY(cuda_status(gated_scan(p, true, part, dec, bp.nblk, nullptr, nullptr, nullptr, nullptr, st)));
    }
    return cuda_status(gated_bwd_kv(p, q, k, v, g, gates, dout, part, bp.block_tokens, bp.nblk, up, col, own, dgp, chunks,
                                    dk, dv, dg, st));
}

la_status la_gated_decode_step(const la_desc* desc, const void* q, const void* k, const void* v, const void* g,
                               const float* S, const float* z, float* S_out, float* z_out, void* out, void* stream) {
    if (desc == nullptr) return LA_ERR_INVALID_ARG;
    la_desc d1 = *desc;
    d1.N = 1;  // N is not used by a step
    LA_TRY(check_desc(&d1));
    if (!q || !k || !v || !g || !S || !z || !S_out || !z_out || !out) return LA_ERR_INVALID_ARG;
    for (const void* ptr : {q, k, v, g, static_cast<const void*>(S), static_cast<const void*>(z),
                            static_cast<const void*>(S_out), static_cast<const void*>(z_out),
                            static_cast<const void*>(out)})
        if (!aligned16(ptr)) return LA_ERR_MISALIGNED;
    LA_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    timing_begin(st);
    return cuda_status(gated_decode(to_problem(&d1), q, k, v, g, S, z, S_out, z_out, out, st));
}

size_t la_qk_norm_rope_workspace_size(const la_rope_desc* desc) {
    if (check_rope(desc) != LA_OK) return 0;
    return WS_HEADER + round_up(qk_rope_partials(*desc, device_sms()) * desc->d * sizeof(float), kAlign);
}

la_status la_qk_norm_rope(const la_rope_desc* desc, const void* q, const la_strides* q_strides, const void* k,
                          const la_strides* k_strides, const float* wq, const float* wk, const float* cos,
                          const float* sin, const int32_t* positions, void* q_out, void* k_out, void* stream) {
    LA_TRY(check_rope(desc));
    LA_TRY(check_rope_inputs(*desc, q, q_strides, k, k_strides, wq, wk, cos, sin, positions));
    if (!q_out || !k_out) return LA_ERR_INVALID_ARG;
    if (!aligned16(q_out) || !aligned16(k_out)) return LA_ERR_MISALIGNED;
    LA_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    timing_begin(st);
    return cuda_status(qk_norm_rope(*desc, q, *q_strides, k, *k_strides, wq, wk, cos, sin, positions, q_out, k_out, st));
}

la_status la_qk_norm_rope_backward(const la_rope_desc* desc, const void* q, const la_strides* q_strides, const void* k,
                                   const la_strides* k_strides, const float* wq, const float* wk, const float* cos,
                                   const float* sin, const int32_t* positions, const void* dq_out, const void* dk_out,
                                   void* dq, const la_strides* dq_strides, void* dk, const la_strides* dk_strides,
                                   float* dwq, float* dwk, void* ws, size_t ws_bytes, void* stream) {
    LA_TRY(check_rope(desc));
    LA_TRY(check_rope_inputs(*desc, q, q_strides, k, k_strides, wq, wk, cos, sin, positions));
    if (!dq_out || !dk_out || !dq || !dk || !dq_strides || !dk_strides) return LA_ERR_INVALID_ARG;
    if ((dwq == nullptr) != (dwk == nullptr)) return LA_ERR_INVALID_ARG;
    for (const void* ptr : {dq_out, dk_out, static_cast<const void*>(dq), static_cast<const void*>(dk),
                            static_cast<const void*>(dwq), static_cast<const void*>(dwk)})
        if (!aligned16(ptr)) return LA_ERR_MISALIGNED;
    LA_TRY(check_strides(*desc, *dq_strides, desc->Hq, true));
    LA_TRY(check_strides(*desc, *dk_strides, desc->Hk, true));
    WsLayout L;
    L.total = la_qk_norm_rope_workspace_size(desc);
    LA_TRY(check_ws(L, ws, ws_bytes));
    LA_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    timing_begin(st);
    return cuda_status(qk_norm_rope_backward(*desc, q, *q_strides, k, *k_strides, wq, wk, cos, sin, positions, dq_out,
                                             dk_out, dq, *dq_strides, dk, *dk_strides, dwq, dwk,
                                             at<float>(ws, WS_HEADER), st));
}

la_status la_last_error(void* ws, void* stream, uint32_t* flags_out) {
    if (ws == nullptr) return LA_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t host = 0;
    LA_TRY(cuda_status(cudaMemcpyAsync(&host, ws, sizeof(uint32_t), cudaMemcpyDeviceToHost, st)));
    LA_TRY(cuda_status(cudaMemsetAsync(ws, 0, sizeof(uint32_t), st)));
    LA_TRY(cuda_status(cudaStreamSynchronize(st)));
    if (flags_out) *flags_out = host;
    if (host & tc::FLAG_TIMEOUT) return LA_ERR_TIMEOUT;
    if (host & FLAG_MASK_RANGE) return LA_ERR_MASK_RANGE;
    return LA_OK;
}

}  // extern "C"
