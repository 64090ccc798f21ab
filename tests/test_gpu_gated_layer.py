"""The gated operators together, as a layer calls them: norm and rotation of a
packed projection, gated prefill with its state, steps that go on from it; and
the gradients of the same chain. Tolerances: those of each operator
(test_gpu_gated, test_gpu_qk_rope), added up. Rounding the rotated q and k
changes a feature relu(x) + 1 by at most half a step of itself, a weight and
the denominator by two each; the rotation's fp32 arithmetic adds (d + 16) 2^-23
of at most 1.5 x the row's largest channel, which is below sqrt(d) (norm 1
per channel, weights at most 1), at each of the four."""

import numpy as np
import pytest
import torch

from oracle import gated as G
from kernelized_linear_attention_phi_b200 import binding as la

from gpu_util import DT, f64
from test_gpu_gated import close, gates, roundings, state_tol, upstream
from test_gpu_qk_rope import HALF, draw, tables

pytestmark = pytest.mark.gpu
EPS = 1e-6


def layer(B, N, H, d, dt, seed):
    x = draw((B, N, 3 * H * d), dt, seed)
    q, k, v = (x[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    w = [torch.rand(d, generator=torch.Generator().manual_seed(seed + i)).cuda() for i in (1, 2)]
    return q, k, v, w, gates(B, H, N, dt, seed, docs=1)


def rotated(x, w, cos, sin, at):
    """fp64, [B, H, N, d]."""
    c, s = (np.broadcast_to(f64(t)[at][:, :, None], (*x.shape[:3], t.shape[-1])) for t in (cos, sin))
    return G.norm_rope(f64(x), f64(w), c, s, EPS, False).transpose(0, 2, 1, 3)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_prefill_then_steps(dt, d):
    B, H, N, T = 2, 3, 337, 9
    q, k, v, w, g = layer(B, N + T, H, d, dt, 51)
    cos, sin = tables(1000, d)
    start = torch.tensor([0, 400], dtype=torch.int32, device="cuda")
    at = start[:, None] + torch.arange(N + T, dtype=torch.int32, device="cuda")
    S, z = torch.empty(B, H, d, d, device="cuda"), torch.empty(B, H, d, device="cuda")
    outs = []
    for a, b in [(0, N)] + [(t, t + 1) for t in range(N, N + T)]:
        q1, k1 = la.la_qk_norm_rope(q[:, a:b], k[:, a:b], *w, cos, sin, positions=at[:, a:b].contiguous())
        v1, g1 = v[:, a:b].transpose(1, 2).contiguous(), g[:, :, a:b].contiguous()
        outs.append(la.la_gated_decode_step(q1, k1, v1, g1, S, z) if a else
                    la.la_gated_causal(q1, k1, v1, g1, S_out=S, z_out=z))
    at = at.cpu().numpy()
    Q, K = rotated(q, w[0], cos, sin, at), rotated(k, w[1], cos, sin, at)
    ref, scale = G.heads(G.gated, Q, K, f64(v).transpose(0, 2, 1, 3), f64(g))
    more = HALF[dt] + (d + 16) * 2.0 ** -23 * 1.5 * d ** 0.5
    close("out", torch.cat(outs, 2), ref[0], scale[0], roundings(dt, d, N + T, "relu1", True)[0] + 4.2 * more)
    close("S", S, ref[1], scale[1], 2 * state_tol(dt, d, N + T) + 1.05 * more)
    close("z", z, ref[2], scale[2], 2 * state_tol(dt, d, N + T) + 1.05 * more)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_gradients_of_the_chain(dt, d):
    """Into one packed gradient; the definition is taken at the rotated q and k
    as they were rounded, where the feature map's kink lies for both."""
    B, H, N = 2, 2, 300
    q, k, v, w, g = layer(B, N, H, d, dt, 52)
    cos, sin = tables(N, d // 2)
    q1, k1 = la.la_qk_norm_rope(q, k, *w, cos, sin)
    v1 = v.transpose(1, 2).contiguous()
    dout = upstream(v1, 6)
    dq1, dk1, dv, dg = la.la_gated_causal_backward(q1, k1, v1, g, dout)
    dx = torch.full((B, N, 3 * H * d), float("nan"), device="cuda", dtype=DT[dt])
    into = [dx[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3)]
    _, _, dwq, dwk = la.la_qk_norm_rope_backward(q, k, *w, cos, sin, dq1, dk1, dq=into[0], dk=into[1])
    into[2].copy_(dv.transpose(1, 2))
    assert bool(dx.isfinite().all())

    ref, scale, _ = G.heads(G.gated_backward, f64(q1), f64(k1), f64(v1), f64(g), f64(dout))
    _, tol, tol_v, _ = roundings(dt, d, N, "relu1", True)
    close("dv", into[2], ref[2].transpose(0, 2, 1, 3), scale[2].transpose(0, 2, 1, 3), tol_v)
    own = HALF[dt] + (d + 16) * 2.0 ** -23
    c, s = (np.broadcast_to(f64(t)[None, :, None], (B, N, H, t.shape[-1])) for t in (cos, sin))
    for name, i, x, ww, dw in (("dq", 0, q, w[0], dwq), ("dk", 1, k, w[1], dwk)):
        dy, err = ref[i].transpose(0, 2, 1, 3), tol * scale[i].transpose(0, 2, 1, 3)
        (want, want_w), _ = G.norm_rope_backward(f64(x), f64(ww), c, s, EPS, False, dy)
        # the operator is linear in dy: its scale at dy's error bounds what that error becomes
        _, (at_dy, at_dy_w) = G.norm_rope_backward(f64(x), f64(ww), c, s, EPS, False, np.abs(dy) + err)
        _, (at_err, at_err_w) = G.norm_rope_backward(f64(x), f64(ww), c, s, EPS, False, err)
        assert (np.abs(f64(into[i]) - want) <= own * at_dy + at_err).all(), name
        n = B * N * H
        assert (np.abs(f64(dw) - want_w) <= (d + 16 + n ** 0.5 + 64) * 2.0 ** -23 * at_dy_w + at_err_w).all(), name


@pytest.mark.parametrize("op", ["gated_causal", "gated_causal_bwd", "gated_decode", "qk_norm_rope", "qk_norm_rope_bwd"])
def test_the_profiling_command_runs_them(op, monkeypatch):
    from kernelized_linear_attention_phi_b200 import profile_case
    monkeypatch.setattr("sys.argv", ["profile_case", "--op", op, "--H", "2", "--N", "200", "--iters", "1"])
    profile_case.main()
