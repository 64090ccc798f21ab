"""fp64 definition of gated linear attention and of the query / key norm with
rotation, with the rounding scales their tests need.

TEST INFRASTRUCTURE, like the rest of this package: numpy float64, one head at
a time, no code shared with the library.

Gated linear attention, from the definition as weights of (query, key) pairs:
with D_ij = a_{j+1} ... a_i (1 for j = i, 0 for j > i), a = exp(g), and
A_ij = D_ij phi(q_i) . phi(k_j),
    num_i = sum_j A_ij v_j + (a_0 ... a_i) phi(q_i) S0, den likewise,
    out = num / den or num.
D is built as products (row i from row i - 1), so a closed gate (a = 0) needs
no special case.

A scale is the same expression with every factor's absolute value: a rounding
of relative size u in a factor moves the result by at most u times it.
"""

from __future__ import annotations

import numpy as np

from .backward import phi_grad
from .linear_attention import PHI_RELU1, phi


def decays(g):
    """D [N, N] and the products a_0 ... a_i [N]."""
    a = np.exp(np.asarray(g, np.float64))
    n = len(a)
    D = np.zeros((n, n))
    for i in range(n):
        if i:
            D[i, :i] = D[i - 1, :i] * a[i]
        D[i, i] = 1.0
    return D, np.cumprod(a)


def gated(Q, K, V, g, phi_kind=PHI_RELU1, normalize=True, S0=None, z0=None):
    """One head. Returns out, S, z and their scales."""
    d = Q.shape[1]
    S0 = np.zeros((d, d)) if S0 is None else S0
    z0 = np.zeros(d) if z0 is None else z0
    a, b = phi(Q, phi_kind), phi(K, phi_kind)
    D, pre = decays(g)
    A = D * (a @ b.T)
    num, den = A @ V + pre[:, None] * (a @ S0), A.sum(1) + pre * (a @ z0)
    aa, ab = np.abs(a), np.abs(b)
    out_s = (D * (aa @ ab.T)) @ np.abs(V) + pre[:, None] * (aa @ np.abs(S0))
    out = num
    if normalize:
        out, out_s = num / den[:, None], out_s / np.abs(den)[:, None]
    last = D[-1][:, None]
    S, z = (last * b).T @ V + pre[-1] * S0, (last * b).sum(0) + pre[-1] * z0
    S_s = (last * ab).T @ np.abs(V) + pre[-1] * np.abs(S0)
    z_s = (last * ab).sum(0) + pre[-1] * np.abs(z0)
    return (out, S, z), (out_s, S_s, z_s)


def gated_backward(Q, K, V, g, dO, phi_kind=PHI_RELU1, normalize=True):
    """One head, empty first state. Returns (dq, dk, dv, dg) and their scales."""
    a, b = phi(Q, phi_kind), phi(K, phi_kind)
    aa, ab = np.abs(a), np.abs(b)
    D, _ = decays(g)
    A, Aa = D * (a @ b.T), D * (aa @ ab.T)
    if normalize:
        den = A.sum(1)
        out, out_s = (A @ V) / den[:, None], (Aa @ np.abs(V)) / np.abs(den)[:, None]
        gn = dO / den[:, None]
        gden, gden_s = -(gn * out).sum(1), (np.abs(gn) * out_s).sum(1)
    else:
        gn, gden = dO, np.zeros(len(Q))
        gden_s = gden
    dP, dPa = gn @ V.T + gden[:, None], np.abs(gn) @ np.abs(V).T + gden_s[:, None]

    def rect(M):
        """sum of M[t:, :t] for every t (sums of the rectangle itself, no differences)."""
        R = np.cumsum(M[::-1], axis=0)[::-1].cumsum(axis=1)
        return np.array([R[t, t - 1] if t else 0.0 for t in range(len(M))])

    sq, sk = phi_grad(Q, phi_kind), phi_grad(K, phi_kind)
    grads = (sq * ((D * dP) @ b), sk * ((D * dP).T @ a), A.T @ gn, rect(A * dP))
    pairs = Aa * dPa
    scales = (np.abs(sq) * ((D * dPa) @ ab), np.abs(sk) * ((D * dPa).T @ aa), Aa.T @ np.abs(gn), rect(pairs))
    # what the pairs of a token's surroundings add up to: fp32 sums over a
    # chunk leave 2^-24 of it
    return grads, scales, pairs.sum(1) + pairs.sum(0)


def heads(fn, *arrays, **kw):
    """fn over the leading [B, H] axes of every array; nested tuples of stacked results."""
    B, H = arrays[0].shape[:2]
    res = [fn(*(x[b, h] for x in arrays), **{n: (v[b, h] if isinstance(v, np.ndarray) else v) for n, v in kw.items()})
           for b in range(B) for h in range(H)]

    def stack(parts):
        if isinstance(parts[0], tuple):
            return tuple(stack([p[i] for p in parts]) for i in range(len(parts[0])))
        return np.stack(parts).reshape(B, H, *np.shape(parts[0]))

    return stack(res)


def rotate(u, cos, sin, interleaved, back=False):
    """R u (or R^T u) for rows u [..., d] with cos, sin [..., rot / 2]."""
    half = cos.shape[-1]
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = u.copy()
    s = -sin if back else sin
    y[..., one] = u[..., one] * cos - u[..., two] * s
    y[..., two] = u[..., two] * cos + u[..., one] * s
    return y


def norm_rope(x, w, cos, sin, eps, interleaved):
    """Rows x [..., d], one rotation per row."""
    r = (np.mean(x * x, -1, keepdims=True) + eps) ** -0.5
    return rotate(x * r * w, cos, sin, interleaved)


def norm_rope_backward(x, w, cos, sin, eps, interleaved, dy):
    """Returns dx, dw (summed over the rows), and their scales."""
    r = (np.mean(x * x, -1, keepdims=True) + eps) ** -0.5
    n = x * r
    v = rotate(dy, cos, sin, interleaved, back=True)
    half = cos.shape[-1]
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    v_s = np.abs(dy)
    v_s[..., two] = np.abs(dy)[..., two] * np.abs(cos) + np.abs(dy)[..., one] * np.abs(sin)
    v_s[..., one] = np.abs(dy)[..., one] * np.abs(cos) + np.abs(dy)[..., two] * np.abs(sin)
    dn, dn_s = v * w, v_s * np.abs(w)
    axes = tuple(range(x.ndim - 1))
    dx = r * (dn - n * np.mean(dn * n, -1, keepdims=True))
    dx_s = r * (dn_s + np.abs(n) * np.mean(dn_s * np.abs(n), -1, keepdims=True))
    return (dx, (v * n).sum(axes)), (dx_s, (v_s * np.abs(n)).sum(axes))
