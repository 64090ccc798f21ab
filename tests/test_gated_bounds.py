"""The norm-wise bounds of the gated tests (gated_bounds.py), on the CPU: their
exact side is the oracle, and they reject what an entry-wise bound in absolute
values lets through."""

import numpy as np
import pytest
import torch

import gated_bounds as GB
from oracle import gated as G

MODES = [("relu1", True), ("relu1", False), ("identity", False), ("elu1", True)]


def draw(N, d, seed, kind, H=2):
    gen = torch.Generator().manual_seed(seed)
    s = d ** -0.5 if kind == "identity" else 1.0
    q, k, v, do = (torch.randn(1, H, N, d, generator=gen).mul(s).bfloat16().double() for _ in range(4))
    g = (-torch.exp(torch.randn(1, H, N, generator=gen)) / 30).bfloat16().double()
    return q, k, v, g, do / s


@pytest.mark.parametrize("kind,normalize", MODES)
def test_the_exact_side_is_the_oracle(kind, normalize):
    q, k, v, g, do = draw(150, 8, 3, kind)
    g[0, 1, 70] = float("-inf")
    a = [x.numpy() for x in (q, k, v, g)]
    ref = G.heads(G.gated, *a, phi_kind=kind, normalize=normalize)[0][0]
    out = GB.chunked(q, k, v, g, kind=kind, normalize=normalize)
    np.testing.assert_allclose(out.numpy(), ref, rtol=1e-9, atol=1e-11)
    ref = G.heads(G.gated_backward, *a, do.numpy(), phi_kind=kind, normalize=normalize)[0]
    for x, y in zip(GB.chunked(q, k, v, g, do, kind=kind, normalize=normalize), ref):
        np.testing.assert_allclose(x.numpy(), y, rtol=1e-8, atol=1e-9)
    r = np.random.default_rng(1)
    S0, z0 = r.standard_normal((1, 2, 8, 8)), 5 + r.random((1, 2, 8))
    ref = G.heads(G.gated, *a, phi_kind=kind, normalize=normalize, S0=S0, z0=z0)[0][0]
    out = GB.chunked(q, k, v, g, kind=kind, normalize=normalize, S0=torch.tensor(S0), z0=torch.tensor(z0))
    np.testing.assert_allclose(out.numpy(), ref, rtol=1e-9, atol=1e-10)


@pytest.mark.parametrize("kind,normalize", MODES)
def test_what_the_bounds_reject(kind, normalize):
    """A dg of zeros, gradients without what blocks give to one another, a
    result off by 2 %, a NaN."""
    q, k, v, g, do = draw(900, 64, 5, kind, H=1)
    kw = dict(kind=kind, normalize=normalize)
    ref, like = GB.allowances("bf16", q, k, v, g, do, **kw)
    # the chunks' parts of the whole without those of 15 chunks' surroundings
    none = GB.chunked(q, k, v, g, do, cross=False, **kw)
    for i, (r, l) in enumerate(zip(ref, like)):
        factor = 3 if i == 3 else 2
        assert GB.excess(l, r, l, factor, 900) <= 0.51
        assert GB.excess(torch.zeros_like(r), r, l, factor, 900) > 5, i
        assert GB.excess(none[i], r, l, factor, 900) > 2, i
        assert GB.excess(r * 1.02, r, l, factor, 900) > 1 or i == 3
        bad = r.clone()
        bad.view(-1)[7] = float("nan")
        assert GB.excess(bad, r, l, factor, 900) == float("inf")
    ref, like = GB.allowances("bf16", q, k, v, g, **kw)
    assert GB.excess(GB.chunked(q, k, v, g, cross=False, **kw), ref, like, 2, 128) > 2
    assert GB.excess(ref * 1.01, ref, like, 2, 128) > 1
