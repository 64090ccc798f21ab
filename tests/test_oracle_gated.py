"""The fp64 definitions behind the gated and norm / rotation tests, pinned on the
CPU: against the ungated oracle, the step-by-step recurrence, differences of
the forward definition, and torch autograd."""

import numpy as np
import pytest
import torch

import oracle
from oracle import gated as G

MODES = [("relu1", True), ("relu1", False), ("identity", False), ("elu1", True)]


def _draw(n, d, seed, closed=()):
    r = np.random.default_rng(seed)
    q, k, v, do = (r.standard_normal((n, d)) for _ in range(4))
    g = -np.exp(r.standard_normal(n)) / 3
    g[list(closed)] = -np.inf
    return q, k, v, g, do


@pytest.mark.parametrize("phi,normalize", MODES)
def test_open_gates_are_the_causal_form(phi, normalize):
    q, k, v, _, do = _draw(23, 5, 1)
    (out, S, z), _ = G.gated(q, k, v, np.zeros(23), phi, normalize)
    np.testing.assert_allclose(out, oracle.causal(q, k, v, phi, normalize)[0], rtol=1e-10, atol=1e-12)
    S_ref, z_ref = oracle.kv_summary(k, v, phi)
    np.testing.assert_allclose(S, S_ref, atol=1e-12)
    np.testing.assert_allclose(z, z_ref, atol=1e-12)
    grads, _, _ = G.gated_backward(q, k, v, np.zeros(23), do, phi, normalize)
    ref = oracle.backward_dense(q, k, v, do, "causal", phi_kind=phi, normalize=normalize)
    for a, b in zip(grads[:3], ref[:3]):
        np.testing.assert_allclose(a, b, atol=1e-11)


@pytest.mark.parametrize("phi,normalize", MODES)
def test_matches_the_recurrence_from_a_state(phi, normalize):
    n, d = 17, 4
    q, k, v, g, _ = _draw(n, d, 2, closed=(9,))
    r = np.random.default_rng(3)
    S0, z0 = r.standard_normal((d, d)), 5 + r.random(d)
    (out, S, z), _ = G.gated(q, k, v, g, phi, normalize, S0, z0)
    s, y = S0.copy(), z0.copy()
    for t in range(n):
        a, b = oracle.phi(q[t], phi), oracle.phi(k[t], phi)
        s = np.exp(g[t]) * s + np.outer(b, v[t])
        y = np.exp(g[t]) * y + b
        np.testing.assert_allclose(out[t], a @ s / (a @ y) if normalize else a @ s, atol=1e-11)
    np.testing.assert_allclose(S, s, atol=1e-12)
    np.testing.assert_allclose(z, y, atol=1e-12)


@pytest.mark.parametrize("phi,normalize", MODES)
def test_gradients_are_the_differences_of_the_forward(phi, normalize):
    n, d = 9, 3
    q, k, v, g, do = _draw(n, d, 4, closed=(5,))
    grads, scales, _ = G.gated_backward(q, k, v, g, do, phi, normalize)
    h = 1e-6
    for which in range(4):
        x = (q, k, v, g)[which]
        num = np.zeros_like(x)
        for i in np.ndindex(*x.shape):
            if not np.isfinite(x[i]):
                continue
            loss = []
            for s in (h, -h):
                y = [q, k, v, g]
                y[which] = x.copy()
                y[which][i] += s
                loss.append(((G.gated(*y, phi, normalize)[0][0]) * do).sum())
            num[i] = (loss[0] - loss[1]) / (2 * h)
        np.testing.assert_allclose(grads[which], num, atol=2e-7)
        assert (scales[which] >= np.abs(grads[which]) - 1e-12).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_and_rotation_against_autograd(interleaved, rot):
    r = np.random.default_rng(5)
    n, d, eps = 6, 8, 1e-3
    x, dy, w = r.standard_normal((n, d)), r.standard_normal((n, d)), 1 + 0.1 * r.standard_normal(d)
    ang = r.standard_normal((n, rot // 2))
    y = G.norm_rope(x, w, np.cos(ang), np.sin(ang), eps, interleaved)
    tx, tw = (torch.tensor(t, requires_grad=True) for t in (x, w))
    u = tx * (tx.square().mean(-1, keepdim=True) + eps).rsqrt() * tw
    pairs = u[:, :rot].reshape(n, rot // 2, 2) if interleaved else u[:, :rot].reshape(n, 2, rot // 2).transpose(1, 2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * torch.polar(
        torch.ones(n, rot // 2, dtype=torch.float64), torch.tensor(ang))) if rot else pairs
    flat = turned.reshape(n, rot) if interleaved else turned.transpose(1, 2).reshape(n, rot)
    ref = torch.cat([flat, u[:, rot:]], 1)
    np.testing.assert_allclose(y, ref.detach().numpy(), atol=1e-12)
    ref.backward(torch.tensor(dy))
    (dx, dw), (dx_s, dw_s) = G.norm_rope_backward(x, w, np.cos(ang), np.sin(ang), eps, interleaved, dy)
    np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-12)
    assert (dx_s >= np.abs(dx) - 1e-12).all() and (dw_s >= np.abs(dw) - 1e-12).all()
