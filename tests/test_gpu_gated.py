"""Gated linear attention on the GPU (la_gated_causal, its gradients, the decode
step) against the fp64 definition.

Tolerances count roundings. u is half a step of the type (bf16 2^-8); an
entry's error is at most R u times its scale, the same expression in absolute
values, with R the roundings on the longest way to it (1.05 R for the products
of errors). With p = 2 for a feature map that rounds phi(q) and phi(k), else 0:
  out  p (features) + 1 (weights or S) + p (denominator) + 1 (result)
  dq   weights' sum p, out.dout 2p + 1, the pair's weight 1, phi(k) p / 2, result 1
       (unnormalized: 1 + p / 2 + 1); dk the same
  dv   p (weights) + p (denominator) + 1 + 1
  dg   pair p, its gradient 3p + 1, state 1, phi(k) p / 2, result 1
fp32 keeps 2^-22 in a product and 2^-23 in an addition to an accumulator; the
longest way has 3 (d + N) / 8 additions, some 64 other operations, and at most
three such sums in a row. A state's terms keep 24 bits (fp32: 2^-22 of a
product) in fp32 sums. fp32 sums over a chunk leave 2^-15 of its pairs in dg whatever dg is."""

import numpy as np
import pytest
import torch

from oracle import gated as G
from kernelized_linear_attention_phi_b200 import binding as la

from gpu_util import DT, f64, qkv

pytestmark = pytest.mark.gpu

MODES = [("relu1", True), ("relu1", False), ("identity", False), ("elu1", True)]
U = 2.0 ** -8


def roundings(dt, d, N, phi, normalize):
    """Relative error per result: out, dq/dk, dv, dg."""
    if dt == "f32":
        return (3 * (3 * (d + N) / 8 + 64) * 2.0 ** -23,) * 4
    p = 0 if phi == "identity" else 2
    n = int(normalize)
    out = p + 1 + n * p + 1
    dq = n * (p + 2 * p + 1) + 1 + p / 2 + 1
    dv = p + n * p + 2
    dg = p + n * (3 * p + 1) + 1 + p / 2 + 1
    return tuple(1.05 * r * U for r in (out, dq, dv, dg))


def state_tol(dt, d, N):
    return 3 * (d + N) / 8 * 2.0 ** -23 + 2.0 ** -20


def gates(B, H, N, dt, seed, docs=0, span=30.0):
    g = torch.Generator().manual_seed(seed + 77)
    x = -torch.exp(torch.randn(B, H, N, generator=g)) / span
    if docs and N > 1:
        at = torch.randint(1, N, (B, docs), generator=g)
        x.scatter_(2, at[:, None].expand(B, H, docs), float("-inf"))
    return x.to(device="cuda", dtype=DT[dt])


def inputs(B, H, N, d, dt, phi, seed, **kw):
    q, k, v = qkv(B, H, N, d, dt, seed=seed, sigma=d ** -0.5 if phi == "identity" else 1.0)
    return q, k, v, gates(B, H, N, dt, seed, **kw)


def upstream(q, seed):
    g = torch.Generator().manual_seed(seed + 4000)
    return torch.randn(q.shape, generator=g).to(device="cuda", dtype=q.dtype)


def some_state(B, H, d, phi, seed):
    g = torch.Generator().manual_seed(seed + 9000)
    S = torch.randn(B, H, d, d, generator=g) * 4
    z = torch.rand(B, H, d, generator=g) * 20 + 20
    return S.cuda(), z.cuda()


def close(name, got, ref, scale, tol, floor=0.0):
    err = np.abs(f64(got) - ref)
    worst = (err - tol * scale - floor).max()
    assert np.isfinite(f64(got)).all(), name
    assert worst <= 1e-30, (name, worst, (err / (scale + 1e-30)).max(), tol)


def check_forward(q, k, v, g, dt, phi, normalize, state=None):
    B, H, N, d = q.shape
    S, z = torch.full((B, H, d, d), np.nan, device="cuda"), torch.full((B, H, d), np.nan, device="cuda")
    kw = {} if state is None else {"S_in": state[0], "z_in": state[1]}
    ws = la.workspace(la.make_desc(B, H, N, d, q.dtype, phi, normalize), "gated_causal")  # its error word is checked afterwards
    out = la.la_gated_causal(q, k, v, g, S_out=S, z_out=z, phi=phi, normalize=normalize, ws=ws, **kw)
    alone = la.la_gated_causal(q, k, v, g, phi=phi, normalize=normalize, **kw)
    kw = {} if state is None else {"S0": f64(state[0]), "z0": f64(state[1])}
    ref, scale = G.heads(G.gated, f64(q), f64(k), f64(v), f64(g), phi_kind=phi, normalize=normalize, **kw)
    # a call that returns its state forms it from more bits: the outputs of the
    # two calls may differ in their last place
    for name, o in (("out", out), ("out without a state", alone)):
        close(name, o, ref[0], scale[0], roundings(dt, d, N, phi, normalize)[0])
    close("S", S, ref[1], scale[1], state_tol(dt, d, N))
    close("z", z, ref[2], scale[2], state_tol(dt, d, N))
    return out, S, z


def check_backward(q, k, v, g, dt, phi, normalize, seed=0):
    B, H, N, d = q.shape
    dout = upstream(q, seed)
    ws = la.workspace(la.make_desc(B, H, N, d, q.dtype, phi, normalize), "gated_causal_bwd")
    got = la.la_gated_causal_backward(q, k, v, g, dout, phi=phi, normalize=normalize, ws=ws)
    ref, scale, around = G.heads(G.gated_backward, f64(q), f64(k), f64(v), f64(g), f64(dout), phi_kind=phi,
                                 normalize=normalize)
    _, dq, dv, dg = roundings(dt, d, N, phi, normalize)
    close("dq", got[0], ref[0], scale[0], dq)
    close("dk", got[1], ref[1], scale[1], dq)
    close("dv", got[2], ref[2], scale[2], dv)
    window = np.stack([around[..., max(0, t - 64):t + 64].sum(-1) for t in range(N)], -1)
    close("dg", got[3], ref[3], scale[3], dg, floor=2.0 ** -15 * window)
    assert (f64(got[3])[np.isneginf(f64(g))] == 0).all()
    return got


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("N", [1, 2, 31, 64, 65, 700])
@pytest.mark.parametrize("phi,normalize", MODES)
def test_forward(dt, d, N, phi, normalize):
    check_forward(*inputs(1, 2, N, d, dt, phi, seed=N + d), dt, phi, normalize)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("N", [1, 2, 33, 64, 127, 700])
@pytest.mark.parametrize("phi,normalize", MODES)
def test_gradients(dt, d, N, phi, normalize):
    check_backward(*inputs(1, 2, N, d, dt, phi, seed=N + 3 * d), dt, phi, normalize)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("N", [1, 100, 600])
def test_forward_from_a_state_and_closed_gates(dt, d, N):
    q, k, v, g = inputs(2, 2, N, d, dt, "elu1", seed=5, docs=3)
    check_forward(q, k, v, g, dt, "elu1", True, some_state(2, 2, d, "elu1", 6))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 64, 128])
def test_gradients_with_closed_gates(dt, d):
    check_backward(*inputs(2, 2, 600, d, dt, "relu1", seed=8, docs=6), dt, "relu1", True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("span", [0.02, 2e4])
def test_fast_and_slow_decay(dt, span):
    """Gates that forget at once (sums of logs in the thousands per chunk) and
    gates that keep nearly all: neither overflows nor loses its differences."""
    for d in (64, 128):
        t = inputs(1, 2, 500, d, dt, "relu1", seed=9, span=span)
        check_forward(*t, dt, "relu1", True)
        check_backward(*t, dt, "relu1", True)


def test_slow_gate_behind_a_closed_one():
    """Decays behind a closed gate are not blurred by its size: the same tokens
    give the same results with and without a prefix that the gate cuts off."""
    q, k, v, g = inputs(1, 1, 60, 64, "f32", "relu1", seed=10, span=500.0)
    full = [torch.cat([x, x], 2) for x in (q, k, v, g)]
    full[3][:, :, 60] = float("-inf")
    full[3][:, :, 30:50] = -1e4
    a = la.la_gated_causal(q, k, v, g)
    b = la.la_gated_causal(*full)[:, :, 60:]
    assert float((a - b).abs().max()) <= 64 * 2.0 ** -23 * float(a.abs().max())


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_gates_that_amplify(dt, d):
    """Positive log-gates, up to a growth of e^40 over the row."""
    q, k, v, g = inputs(1, 2, 400, d, dt, "relu1", seed=16)
    g = (-g * 0.8).to(g.dtype).clamp(max=0.25)
    check_forward(q, k, v, g, dt, "relu1", True)
    check_backward(q, k, v, g, dt, "relu1", True)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_nan_gate_reaches_its_own_head_from_there_on(dt, d, bad):
    q, k, v, g = inputs(1, 2, 500, d, dt, "relu1", seed=17)
    ref, scale = G.heads(G.gated, f64(q), f64(k), f64(v), f64(g), phi_kind="relu1", normalize=True)
    want = la.la_gated_causal(q, k, v, g)
    g[0, 1, 333] = bad
    got = la.la_gated_causal(q, k, v, g)
    assert torch.equal(got[0, 0], want[0, 0])
    # its chunk takes the decays per pair: other roundings, within the same bounds
    close("out", got[0, 1, :333], ref[0][0, 1, :333], scale[0][0, 1, :333], roundings(dt, d, 500, "relu1", True)[0])
    assert bool(got[0, 1, 333:].isnan().all())


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 16), ("f32", 64)])
@pytest.mark.parametrize("normalize", [True, False])
def test_a_nan_in_q_k_or_v_is_not_lost(dt, d, normalize):
    """NaN as the device makes it (all bits set), which must pass the products'
    parts. Up to 63 tokens in front of it may share its tile, none before them."""
    phi = "elu1" if normalize else "identity"
    q, k, v, g = inputs(1, 2, 500, d, dt, phi, seed=18)
    nan = torch.full((), 0x7FFFFFFF, dtype=torch.int32, device="cuda").view(torch.float32).to(q.dtype)
    for i, x in enumerate((q, k, v)):
        x = x.clone()
        x[0, 1, 333, 5] = nan
        qkv_ = [x if j == i else y for j, y in enumerate((q, k, v))]
        out = la.la_gated_causal(*qkv_, g, phi=phi, normalize=normalize)[0]
        assert not out[0].isnan().any() and not out[1, :270].isnan().any()
        if i == 0:
            assert bool(out[1, 333].isnan().all()) and not out[1, 397:].isnan().any()
        elif i == 1:
            assert bool(out[1, 333:].isnan().all())
        else:
            assert bool(out[1, 333:, 5].isnan().all())


@pytest.mark.parametrize("phi,normalize", [("relu1", True), ("identity", False)])
def test_gradients_at_d128_with_long_blocks(phi, normalize):
    """40 heads of 900 tokens: blocks of 300, whose states go through the tensor
    cores in both directions."""
    check_backward(*inputs(2, 20, 900, 128, "bf16", phi, seed=18, docs=2), "bf16", phi, normalize)


def test_many_heads_in_one_block_and_few_in_many():
    check_forward(*inputs(3, 160, 130, 16, "bf16", "relu1", seed=12), "bf16", "relu1", True)
    check_backward(*inputs(1, 1, 1500, 64, "bf16", "relu1", seed=13), "bf16", "relu1", True)
    check_forward(*inputs(1, 1, 1500, 128, "bf16", "identity", seed=14), "bf16", "identity", False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pieces_and_steps_continue_a_row(dt):
    """A prompt in two pieces (state updated in place), then steps: the same
    states and outputs as the whole row."""
    B, H, N, d = 2, 3, 300, 64
    q, k, v, g = inputs(B, H, N, d, dt, "relu1", seed=15)
    ref, scale = G.heads(G.gated, f64(q), f64(k), f64(v), f64(g))
    S, z = torch.zeros(B, H, d, d, device="cuda"), torch.zeros(B, H, d, device="cuda")
    outs = []
    for a, b in ((0, 130), (130, 290)):
        part = [x[:, :, a:b].contiguous() for x in (q, k, v, g)]
        outs.append(la.la_gated_causal(*part, S_in=S, z_in=z, S_out=S, z_out=z))
    for t in range(290, N):
        part = [x[:, :, t:t + 1].contiguous() for x in (q, k, v, g)]
        outs.append(la.la_gated_decode_step(*part, S, z))
    close("out", torch.cat(outs, 2), ref[0], scale[0], roundings(dt, d, N, "relu1", True)[0])
    close("S", S, ref[1], scale[1], 2 * state_tol(dt, d, N))
    close("z", z, ref[2], scale[2], 2 * state_tol(dt, d, N))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("phi,normalize", MODES)
def test_step(dt, d, phi, normalize):
    B, H = 3, 5
    q, k, v, g = inputs(B, H, 1, d, dt, phi, seed=d)
    g[0, 0] = float("-inf")
    S, z = some_state(B, H, d, phi, 1)
    S1, z1 = torch.empty_like(S), torch.empty_like(z)
    keep = S.clone(), z.clone()
    out = la.la_gated_decode_step(q, k, v, g, S, z, S_out=S1, z_out=z1, phi=phi, normalize=normalize)
    assert torch.equal(S, keep[0]) and torch.equal(z, keep[1])
    ref, scale = G.heads(G.gated, f64(q), f64(k), f64(v), f64(g), phi_kind=phi, normalize=normalize, S0=f64(S), z0=f64(z))
    tol = (d + 16) * 2.0 ** -23
    close("out", out, ref[0], scale[0], 2 * tol + (U if dt == "bf16" else 0))
    close("S", S1, ref[1], scale[1], tol)
    close("z", z1, ref[2], scale[2], tol)
    again = la.la_gated_decode_step(q, k, v, g, S, z, phi=phi, normalize=normalize)
    assert torch.equal(again, out) and torch.equal(S, S1) and torch.equal(z, z1)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nothing_is_written_outside(dt):
    """Outputs inside larger buffers: what lies around them stays."""
    for N, d in ((1, 16), (77, 64), (333, 128)):
        q, k, v, g = inputs(1, 3, N, d, dt, "relu1", seed=20)

        def boxed(shape, dtype):
            n = int(np.prod(shape))
            pad = 64
            buf = torch.full((n + 2 * pad + 16,), 7.0, device="cuda", dtype=dtype)
            return buf, buf[pad:pad + n].view(shape), pad, n

        boxes = [boxed(q.shape, q.dtype) for _ in range(4)] + [boxed((1, 3, d, d), torch.float32), boxed((1, 3, d), torch.float32)]
        dgb = boxed(g.shape, g.dtype)
        la.la_gated_causal(q, k, v, g, out=boxes[0][1], S_out=boxes[4][1], z_out=boxes[5][1])
        la.la_gated_causal_backward(q, k, v, g, upstream(q, 1), dq=boxes[1][1], dk=boxes[2][1], dv=boxes[3][1], dg=dgb[1])
        for buf, _, pad, n in boxes + [dgb]:
            assert bool((buf[:pad] == 7).all()) and bool((buf[pad + n:] == 7).all())


def test_repeated_calls_are_identical():
    q, k, v, g = inputs(1, 3, 900, 64, "bf16", "relu1", seed=21)
    dout = upstream(q, 2)
    a, b = (la.la_gated_causal_backward(q, k, v, g, dout) for _ in range(2))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_capture_replay_and_other_streams():
    q, k, v, g = inputs(1, 2, 700, 64, "bf16", "relu1", seed=22)
    dout = upstream(q, 3)
    want = la.la_gated_causal(q, k, v, g)
    grads = la.la_gated_causal_backward(q, k, v, g, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = la.la_gated_causal(q, k, v, g, stream=side)
    got_grads = la.la_gated_causal_backward(q, k, v, g, dout, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(got_grads, grads))
    out = torch.empty_like(q)
    ws = la.workspace(la._desc_of(q, "relu1", True), "gated_causal")
    wsb = la.workspace(la._desc_of(q, "relu1", True), "gated_causal_bwd")
    res = [torch.empty_like(x) for x in grads]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        la.la_gated_causal(q, k, v, g, out=out, ws=ws)
        la.la_gated_causal_backward(q, k, v, g, dout, *res, ws=wsb)
    for _ in range(2):
        for x in (out, *res):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(res, grads))


def test_the_binding_refuses_what_does_not_fit():
    q, k, v, g = inputs(1, 2, 8, 64, "bf16", "relu1", seed=30)
    S, z = some_state(1, 2, 64, "relu1", 1)
    good = dict(q=q, k=k, v=v, g=g)
    for bad in (dict(k=k.float()), dict(v=v[:, :, :4].contiguous()), dict(g=g.float()), dict(g=g[:, :, :4].contiguous()),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(g=g.cpu()), dict(S_in=S, z_in=z.double()),
                dict(S_out=S[:, :, :, :32], z_out=z), dict(out=torch.empty_like(q).float()),
                dict(ws=torch.zeros(512, device="cuda"))):
        with pytest.raises((ValueError, la.LaError)):
            la.la_gated_causal(**{**good, **bad})
    with pytest.raises(ValueError):
        la.la_gated_causal_backward(q, k, v, g, upstream(q, 1).float())
    with pytest.raises(la.LaError, match="UNSUPPORTED"):
        la.la_gated_causal(q, k, v, g, phi="identity", normalize=True)
    with pytest.raises(la.LaError, match="WORKSPACE"):
        la.la_gated_causal_backward(q, k, v, g, q, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(la.LaError, match="MISALIGNED"):
        flat = torch.zeros(q.numel() + 8, device="cuda", dtype=q.dtype)
        la.la_gated_causal(flat[1:1 + q.numel()].view(q.shape), k, v, g)
