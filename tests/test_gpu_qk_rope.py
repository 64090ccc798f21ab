"""Norm and rotation of queries and keys on the GPU against the fp64
definition. An entry errs by at most half a step of its type once (the result)
and by fp32 arithmetic (sums of d terms, rsqrt, the rotation): (d + 16) 2^-23
of the same expression in absolute values."""

import numpy as np
import pytest
import torch

from oracle import gated as G
from kernelized_linear_attention_phi_b200 import binding as la

from gpu_util import DT, f64

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def tables(rows, rot):
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    return ang.cos().float().cuda(), ang.sin().float().cuda()


def draw(shape, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(device="cuda", dtype=DT[dt])


def packed(B, N, Hq, Hk, d, dt, seed):
    x = draw((B, N, (Hq + 2 * Hk) * d), dt, seed)
    return x[..., :Hq * d].unflatten(-1, (Hq, d)), x[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))


def check(q, k, wq, wk, cos, sin, at, interleaved, dt, eps=1e-6):
    B, N, Hq, d = q.shape
    Hk = k.shape[2]
    dyq, dyk = draw((B, Hq, N, d), dt, 91), draw((B, Hk, N, d), dt, 92)
    got = la.la_qk_norm_rope(q, k, wq, wk, cos, sin, positions=at, eps=eps, interleaved=interleaved)
    grads = la.la_qk_norm_rope_backward(q, k, wq, wk, cos, sin, dyq, dyk, positions=at, eps=eps, interleaved=interleaved)
    pos = np.arange(N)[None].repeat(B, 0) if at is None else at.cpu().numpy()
    if cos is None:
        c = s = np.zeros((B, N, 1, 0))
    else:
        c, s = f64(cos)[pos][:, :, None], f64(sin)[pos][:, :, None]
    tol = HALF[dt] + (d + 16) * 2.0 ** -23
    for i, (x, w, dy) in enumerate(((q, wq, dyq), (k, wk, dyk))):
        ww = np.ones(d) if w is None else f64(w)
        cc, ss = (np.broadcast_to(t, (*x.shape[:3], t.shape[-1])) for t in (c, s))
        y = G.norm_rope(f64(x), ww, cc, ss, eps, interleaved)
        u = np.abs(G.norm_rope(f64(x), ww, cc[..., :0], ss[..., :0], eps, interleaved))
        scale = np.maximum(np.abs(y), 1.5 * np.abs(u).max(-1, keepdims=True))
        err = np.abs(f64(got[i]).transpose(0, 2, 1, 3) - y)
        assert (err <= HALF[dt] * np.abs(y) + (d + 16) * 2.0 ** -23 * scale).all(), (i, err.max())
        (dx, dw), (dx_s, dw_s) = G.norm_rope_backward(f64(x), ww, cc, ss, eps, interleaved, f64(dy).transpose(0, 2, 1, 3))
        assert (np.abs(f64(grads[i]) - dx) <= tol * dx_s).all(), i
        if w is not None:
            n = B * N * x.shape[2]
            assert (np.abs(f64(grads[2 + i]) - dw) <= (d + 16 + n ** 0.5 + 64) * 2.0 ** -23 * dw_s).all(), i
    return got, grads


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_packed_projection(dt, d, interleaved):
    for B, N, Hq, Hk, rot in ((1, 1, 1, 1, d), (2, 37, 6, 2, d), (3, 130, 5, 5, 16), (64, 1, 4, 4, d)):
        q, k = packed(B, N, Hq, Hk, d, dt, seed=d + N)
        wq, wk = 1 + 0.2 * draw((d,), "f32", 3), 1 + 0.2 * draw((d,), "f32", 4)
        cos, sin = tables(300, rot)
        at = torch.randint(0, 300, (B, N), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
        check(q, k, wq, wk, cos, sin, at, interleaved, dt)
        check(q, k, wq, wk, cos, sin, None, interleaved, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_other_layouts_no_weights_no_rotation(dt):
    B, H, N, d = 2, 3, 21, 64
    base = draw((B, H, N, d), dt, 6)
    q = base.transpose(1, 2)                      # [B, N, H, d] view of [B, H, N, d]
    k = draw((B, N, 1, d), dt, 7).expand(B, N, 4, d)  # one key head read by four
    cos, sin = tables(64, 32)
    check(q, k, None, None, cos, sin, None, True, dt)
    check(q, k, None, None, None, None, None, False, dt)


def test_gradients_into_one_packed_buffer():
    B, N, Hq, Hk, d = 2, 50, 4, 2, 32
    q, k = packed(B, N, Hq, Hk, d, "bf16", 8)
    w = torch.ones(d, device="cuda")
    cos, sin = tables(64, d)
    dyq, dyk = draw((B, Hq, N, d), "bf16", 9), draw((B, Hk, N, d), "bf16", 10)
    want = la.la_qk_norm_rope_backward(q, k, w, w, cos, sin, dyq, dyk)
    buf = torch.full((B, N, (Hq + 2 * Hk) * d), 7.0, device="cuda", dtype=torch.bfloat16)
    dq, dk = buf[..., :Hq * d].unflatten(-1, (Hq, d)), buf[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    la.la_qk_norm_rope_backward(q, k, w, w, cos, sin, dyq, dyk, dq=dq, dk=dk)
    assert torch.equal(dq, want[0]) and torch.equal(dk, want[1])
    assert bool((buf[..., (Hq + Hk) * d:] == 7).all())


def test_a_position_outside_the_tables_makes_nan_of_its_rows_only():
    B, N, H, d = 1, 9, 2, 64
    q, k = packed(B, N, H, H, d, "f32", 11)
    cos, sin = tables(16, 32)
    at = torch.arange(N, dtype=torch.int32, device="cuda")[None].contiguous()
    good = la.la_qk_norm_rope(q, k, None, None, cos, sin, positions=at)
    at[0, 3], at[0, 5] = 16, -1
    bad = la.la_qk_norm_rope(q, k, None, None, cos, sin, positions=at)
    rows = torch.ones(N, dtype=torch.bool, device="cuda")
    rows[[3, 5]] = False
    for a, b in zip(good, bad):
        assert torch.equal(a[:, :, rows], b[:, :, rows]) and bool(b[:, :, ~rows].isnan().all())


def test_rows_of_zeros_and_long_tables():
    q = torch.zeros(1, 3, 1, 64, device="cuda")
    cos, sin = tables(1 << 20, 64)
    at = torch.tensor([[0, (1 << 20) - 1, 77777]], dtype=torch.int32, device="cuda")
    y, _ = la.la_qk_norm_rope(q, q, None, None, cos, sin, positions=at)
    assert bool((y == 0).all())
    q = draw((1, 3, 2, 64), "f32", 12)
    check(q, q, None, None, cos, sin, at, False, "f32")


def test_capture_and_replay():
    q, k = packed(2, 40, 4, 4, 64, "bf16", 13)
    w = 1 + 0.1 * draw((64,), "f32", 14)
    cos, sin = tables(64, 64)
    dyq = draw((2, 4, 40, 64), "bf16", 15)
    want = la.la_qk_norm_rope(q, k, w, w, cos, sin)
    grads = la.la_qk_norm_rope_backward(q, k, w, w, cos, sin, dyq, dyq)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = la.la_qk_norm_rope(q, k, w, w, cos, sin)
        got_grads = la.la_qk_norm_rope_backward(q, k, w, w, cos, sin, dyq, dyq)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *got_grads), (*want, *grads)))


def test_the_binding_refuses_what_does_not_fit():
    q, k = packed(2, 9, 4, 2, 64, "bf16", 16)
    t, w = torch.zeros(16, 32, device="cuda"), torch.ones(64, device="cuda")
    good = dict(q=q, k=k, q_weight=w, k_weight=w, cos=t, sin=t)
    la.la_qk_norm_rope(**good)
    for bad in (dict(k=k[:, :5]), dict(k=k.float()), dict(q=q[0]), dict(sin=None), dict(sin=t[:, :16]), dict(cos=t.double()),
                dict(q_weight=None), dict(q_weight=w[:32]), dict(k_weight=w.bfloat16()),
                dict(cos=torch.zeros(16, 40, device="cuda"), sin=torch.zeros(16, 40, device="cuda")),
                dict(positions=torch.zeros(2, 9, device="cuda")), dict(positions=torch.zeros(9, dtype=torch.int32, device="cuda")),
                dict(q=q.transpose(2, 3)), dict(q_out=torch.empty(2, 9, 4, 64, device="cuda", dtype=q.dtype))):
        with pytest.raises(ValueError):
            la.la_qk_norm_rope(**{**good, **bad})
    with pytest.raises(la.LaError, match="INVALID_ARG"):  # nine tokens, eight rows, no positions
        la.la_qk_norm_rope(q, k, None, None, t[:8], t[:8])
    with pytest.raises(la.LaError, match="UNSUPPORTED"):  # 24 channels turned
        la.la_qk_norm_rope(q, k, None, None, t[:, :12].contiguous(), t[:, :12].contiguous())
    with pytest.raises(ValueError, match="no weights"):
        la.la_qk_norm_rope_backward(q, k, None, None, t, t, torch.empty(2, 4, 9, 64, device="cuda", dtype=q.dtype),
                                    torch.empty(2, 2, 9, 64, device="cuda", dtype=q.dtype), dq_weight=w, dk_weight=w)
    with pytest.raises(la.LaError, match="INVALID_ARG"):  # gradient rows on one another
        dy = torch.zeros(2, 4, 9, 64, device="cuda", dtype=q.dtype)
        la.la_qk_norm_rope_backward(q, q, w, w, t, t, dy, dy, dq=torch.zeros(2, 9, 1, 64, device="cuda", dtype=q.dtype).expand(2, 9, 4, 64))
