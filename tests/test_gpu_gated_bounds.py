"""Gated linear attention on the GPU under norm-wise bounds (gated_bounds.py):
where results would be lost although every entry stays within an entry-wise
bound, and inputs and gates at the ends of the range."""

import pytest
import torch

import gated_bounds as GB
from kernelized_linear_attention_phi_b200 import binding as la

from gpu_util import DT, qkv

pytestmark = pytest.mark.gpu

MODES = [("relu1", True), ("relu1", False), ("identity", False), ("elu1", True)]
KINDS = [("bf16", 16), ("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 16), ("f32", 64), ("f32", 128)]


def inputs(B, H, N, d, dt, phi, seed, span=30.0, sigma=1.0):
    q, k, v = qkv(B, H, N, d, dt, seed=seed, sigma=sigma * (d ** -0.5 if phi == "identity" else 1.0))
    gen = torch.Generator().manual_seed(seed + 77)
    g = (-torch.exp(torch.randn(B, H, N, generator=gen)) / span).to(device="cuda", dtype=DT[dt])
    dout = torch.randn(B, H, N, d, generator=gen).to(device="cuda", dtype=DT[dt])
    return q, k, v, g, dout


def rate(dt, d, lowest):
    """A gate that takes every chunk's sum (of 32 tokens in fp32 with d >= 64, else 64) to 2^lowest."""
    return lowest / 1.4427 / (32 if dt == "f32" and d >= 64 else 64)


def check_out(dt, q, k, v, g, phi, normalize, window=64, **state):
    kw = {n: s.double() for n, s in zip(("S0", "z0"), state.values())}
    ref, like = GB.allowances(dt, *(x.double() for x in (q, k, v, g)), kind=phi, normalize=normalize, **kw)
    out = la.la_gated_causal(q, k, v, g, phi=phi, normalize=normalize, **state)
    x = GB.excess(out.double(), ref, like, 2, window)
    assert x <= 1, x
    return out


def check_gradients(dt, q, k, v, g, dout, phi, normalize, window=128):
    ref, like = GB.allowances(dt, *(x.double() for x in (q, k, v, g, dout)), kind=phi, normalize=normalize)
    got = la.la_gated_causal_backward(q, k, v, g, dout, phi=phi, normalize=normalize)
    x = [GB.excess(a.double(), r, l, 3 if i == 3 else 2, g.shape[2] if i == 3 else window)
         for i, (a, r, l) in enumerate(zip(got, ref, like))]
    assert max(x) <= 1, x
    return got


@pytest.mark.parametrize("dt,d", KINDS)
@pytest.mark.parametrize("phi,normalize", MODES)
def test_norms(dt, d, phi, normalize):
    q, k, v, g, dout = inputs(1, 2, 900, d, dt, phi, seed=d)
    check_out(dt, q, k, v, g, phi, normalize)
    check_gradients(dt, q, k, v, g, dout, phi, normalize)


@pytest.mark.parametrize("phi,normalize", MODES)
def test_norms_of_long_blocks_at_d128(phi, normalize):
    """40 heads of 900 tokens: the gradients' block states on the tensor cores, in both directions."""
    q, k, v, g, dout = inputs(2, 20, 900, 128, "bf16", phi, seed=4)
    check_gradients("bf16", q, k, v, g, dout, phi, normalize)


@pytest.mark.parametrize("dt,d", KINDS)
@pytest.mark.parametrize("phi,normalize", MODES)
@pytest.mark.parametrize("lowest", [-88.0, -50.0, -120.0])
def test_large_values_under_fast_gates(dt, d, phi, normalize, lowest):
    """Values of thousands and an upstream of 65536 under gates that close a chunk by 50 to 120 bits: no
    factor of a decay stands next to a product of tokens for longer than the decay itself."""
    q, k, v, g, dout = inputs(1, 2, 200, d, dt, phi, seed=11, sigma=4000.0 * (d ** 0.5 if phi == "identity" else 1.0))
    g.fill_(rate(dt, d, lowest))
    check_out(dt, q, k, v, g, phi, normalize)
    q, k, v = (x / 32 for x in (q, k, v))
    if phi == "elu1":  # e^-4000 has no digits to compare: features between e^-30 and 125
        q, k = q.clamp(min=-30), k.clamp(min=-30)
    check_gradients(dt, q, k, v, g, dout * 65536, phi, normalize)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 32), ("f32", 64)])
@pytest.mark.parametrize("phi,normalize", MODES)
def test_small_upstream_under_fast_gates(dt, d, phi, normalize):
    """A loss's mean over many tokens makes upstream gradients of 2^-40: a decay of 2^-88 next to them
    leaves fp32's normal range."""
    q, k, v, g, dout = inputs(1, 2, 200, d, dt, phi, seed=12)
    g.fill_(rate(dt, d, -88.0))
    check_gradients(dt, q, k, v, g, dout * 2.0 ** -40, phi, normalize)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_denominators_near_the_largest_float(dt, d):
    """Two tokens that see themselves alone, with phi(q).phi(k) between 2^126 and 2^127: each output is its value."""
    q = torch.full((1, 1, 2, d), 1.125 * 2.0 ** 63 / d ** 0.5, device="cuda").to(DT[dt])
    v = torch.linspace(-0.25, 0.25, 2 * d, device="cuda").view(1, 1, 2, d).to(DT[dt])
    g = torch.full((1, 1, 2), float("-inf"), device="cuda", dtype=DT[dt])
    assert 2.0 ** 126 < float((q.double() * q.double()).sum(-1).max()) < 2.0 ** 127
    out = la.la_gated_causal(q, q, v, g)
    step = torch.finfo(DT[dt]).eps
    assert float((out.double() - v.double()).abs().max()) <= 0.25 * (step if dt == "bf16" else 8 * step)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("phi,normalize", [("relu1", True), ("identity", False)])
@pytest.mark.parametrize("closed", [1, 16, 40, 63])
def test_closed_gates_in_front_inside_the_chunk(dt, d, phi, normalize, closed):
    """Padding in front of a document: `closed` tokens of closed gates, then the document from inside the
    chunk on. Its results are those of the document alone."""
    q, k, v, g, dout = inputs(1, 2, 256, d, dt, phi, seed=13)
    g[:, :, :closed + 1] = float("-inf")
    out = check_out(dt, q, k, v, g, phi, normalize, window=32)
    got = check_gradients(dt, q, k, v, g, dout, phi, normalize)
    alone = [x[:, :, closed:].contiguous() for x in (q, k, v, g, dout)]
    ref, like = GB.allowances(dt, *(x.double() for x in alone[:4]), kind=phi, normalize=normalize)
    assert GB.excess(out[:, :, closed:].double(), ref, like, 2, 32) <= 1
    ref, like = GB.allowances(dt, *(x.double() for x in alone), kind=phi, normalize=normalize)
    for i in range(3):
        assert GB.excess(got[i][:, :, closed:].double(), ref[i], like[i], 2, 128) <= 1


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("length", [2, 4, 13])
def test_rows_of_short_documents(dt, d, length):
    q, k, v, g, dout = inputs(1, 2, 300, d, dt, "relu1", seed=14)
    g[:, :, ::length] = float("-inf")
    check_out(dt, q, k, v, g, "relu1", True)
    check_gradients(dt, q, k, v, g, dout, "relu1", True)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_closed_gates_behind_a_state(dt, d):
    """Documents inside a row that starts from a state."""
    q, k, v, g, _ = inputs(1, 2, 200, d, dt, "relu1", seed=15)
    g[:, :, 5] = g[:, :, 7:30] = float("-inf")
    S = torch.randn(1, 2, d, d, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) * 4
    z = torch.rand(1, 2, d, device="cuda", generator=torch.Generator("cuda").manual_seed(4)) * 20 + 20
    check_out(dt, q, k, v, g, "relu1", True, window=32, S_in=S, z_in=z)


@pytest.mark.parametrize("dt,d", [("bf16", 64), ("bf16", 128), ("f32", 16), ("f32", 64)])
@pytest.mark.parametrize("sign", [0, 1])
@pytest.mark.parametrize("phi,normalize", MODES)
def test_a_nan_of_either_sign_reaches_prompt_step_and_gradients(dt, d, sign, phi, normalize):
    """The same NaN in q or k for every entry point and map (relu as a plain maximum would make 0 of it)."""
    q, k, v, g, dout = inputs(1, 1, 200, d, dt, phi, seed=16)
    word, top = (0x7FC0, 15) if dt == "bf16" else (0x7FC00000, 31)
    nan = torch.tensor(word - (sign << top), dtype=torch.int16 if dt == "bf16" else torch.int32).view(DT[dt]).cuda()
    for i in range(2):
        a = [q.clone(), k.clone(), v, g]
        a[i][0, 0, 150, 5] = nan
        assert bool(a[i][0, 0, 150, 5].isnan()) and bool(a[i][0, 0, 150, 5].signbit()) == bool(sign)
        out = la.la_gated_causal(*a, phi=phi, normalize=normalize)[0, 0]
        assert not out[:128].isnan().any() and bool(out[150].isnan().all())
        assert bool(out[151:].isnan().all()) if i else not out[151:].isnan().any()
        dq, dk, dv, dg = (x[0, 0] for x in la.la_gated_causal_backward(*a, dout, phi=phi, normalize=normalize))
        if normalize:  # the denominator
            assert bool(dq[150].isnan().all())
        elif i == 0:  # every earlier value meets phi(q)
            assert bool(dv[:128].isnan().all())
        else:  # every later query's channel meets phi(k)
            assert bool(dq[150:, 5].isnan().all())
        one = [x[:, :, 150:151].clone() for x in a]
        S, z = torch.zeros(1, 1, d, d, device="cuda"), torch.zeros(1, 1, d, device="cuda")
        assert bool(la.la_gated_decode_step(*one, S, z, phi=phi, normalize=normalize).isnan().all())


@pytest.mark.parametrize("dt,d", KINDS)
@pytest.mark.parametrize("lowest", [-50.0, -88.0, -120.0])
def test_small_features_under_fast_gates(dt, d, lowest):
    """Queries whose features are all some 2^-45 (elu + 1 of -31): a decay next to them must not take them out
    of their type's range."""
    q, k, v, g, dout = inputs(1, 2, 200, d, dt, "elu1", seed=17)
    g.fill_(rate(dt, d, lowest))
    q = (q - 31).clamp(max=-28)
    check_out(dt, q, k, v, g, "elu1", True)
    check_gradients(dt, q, k, v, g, dout, "elu1", True)


@pytest.mark.parametrize("shape,span", [((2, 3, 167, 16), 400.0), ((2, 3, 283, 64), 400.0), ((3, 6, 290, 16), 200.0),
                                        ((1, 9, 2081, 16), 1000.0)])
def test_dg_does_not_carry_the_roundings_of_the_state(shape, span):
    """Identity map, gates that keep hundreds of tokens: dg cancels down from sums over whole states. The
    state's copies in bf16 would all err the same way there; left are the later queries' state as an operand
    and the result's rounding, the very same in the emulation: a quarter more is allowed for fp32 sums."""
    for seed in range(3):
        q, k, v, g, dout = inputs(*shape, "bf16", "identity", seed=30 + seed, span=span)
        args = [x.double() for x in (q, k, v, g, dout)]
        ref, like = GB.allowances("bf16", *args, kind="identity", normalize=False)
        got = la.la_gated_causal_backward(q, k, v, g, dout, phi="identity", normalize=False)
        off = float((got[3].double() - ref[3]).norm() / (like[3] - ref[3]).norm())
        assert off <= 1.25, (seed, off)


@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("phi", ["relu1", "elu1"])
@pytest.mark.parametrize("sigma", [0.1, 0.02])
def test_small_queries_and_keys_keep_their_digits_in_dq(d, phi, sigma):
    """Features next to 1: dq is what is left of sums that all channels share, and 1 + x rounded to bf16
    would have lost most of x."""
    q, k, v, g, dout = inputs(1, 4, 500, d, "bf16", phi, seed=19, sigma=sigma)
    check_gradients("bf16", q, k, v, g, dout, phi, True)


@pytest.mark.parametrize("dt,d", KINDS)
@pytest.mark.parametrize("phi,normalize", MODES)
@pytest.mark.parametrize("gate", [-4.0, -8.0, -14.0])
def test_gradients_under_gates_that_keep_little(dt, d, phi, normalize, gate):
    """Every gate lets through 2 % to a millionth: dg (and dq, dk of a normalized output) are small next to
    what each token has with itself, and come from the pairs of different tokens alone."""
    q, k, v, g, dout = inputs(1, 2, 150, d, dt, phi, seed=20)
    g.fill_(gate)
    check_gradients(dt, q, k, v, g, dout, phi, normalize)
