"""How far the gated kernels may be off, norm by norm: the operators chunk by
chunk in 64 bits, rounded at the places where the kernels round.

``chunked`` with ``exact`` as its rounding is the operator itself; with
``to_bf16`` every operand that the bf16 kernels hold in bf16 is rounded once,
and with ``fp32_noise`` every product is off by up to 2^-21 either way. What
that does to a result's norm is what the kernel's own roundings, which are as
many and as large but fall on other values, do to it; twice that is allowed
(three times for dg, whose entries share their sums' errors).

The two sweeps of the gradients form the products of a pair of tokens each for
itself, so what cancels between them (dg) keeps both sweeps' errors.

In fp32 a product of two-part operands or an exponential is off by up to
2^-22, and a sum of n steps, each rounded to nearest at random, by some
sqrt(n) 2^-24: 2^-22 again for the 16 steps of a product over 256 channels or
tokens. Both together are the 2^-21."""

import torch

CHUNK = 64


def exact(x):
    return x


def to_bf16(x):
    return x.float().bfloat16().double()


def fp32_noise(seed):
    gen = torch.Generator().manual_seed(seed)

    def noise(x):
        u = torch.rand(x.shape, generator=gen, dtype=torch.float64).to(x.device)
        return x * (1 + 2.0 ** -21 * (2 * u - 1))

    return noise


def phi(x, kind):
    if kind == "relu1":
        return x.clamp(min=0) + 1
    return x if kind == "identity" else torch.where(x > 0, x + 1, torch.exp(x.clamp(max=0)))


def slope(x, kind):
    if kind == "relu1":
        return (x > 0).double()
    return torch.ones_like(x) if kind == "identity" else torch.where(x > 0, torch.ones_like(x), torch.exp(x.clamp(max=0)))


def chunked(q, k, v, g, dout=None, kind="relu1", normalize=True, S0=None, z0=None, rnd=exact, bf16=True, cross=True):
    """out, or with dout (dq, dk, dv, dg), of [..., N, d] in float64 tensors.
    bf16: the state goes into the outputs' products rounded once, and into those
    of the gradients' first sweep in two parts. cross = False leaves out what the chunks give
    to one another."""
    lead, (N, d) = q.shape[:-2], q.shape[-2:]
    q, k, v = (x.reshape(-1, N, d) for x in (q, k, v))
    g = g.reshape(-1, N).clamp(min=-1e4)
    H = q.shape[0]
    one = int(kind != "identity")
    prod = exact if bf16 else rnd  # products of bf16 operands are exact in fp32
    S = q.new_zeros(H, d, d) if S0 is None else S0.reshape(H, d, d)
    z = q.new_zeros(H, d) if z0 is None else z0.reshape(H, d)
    spans = [(i, min(N, i + CHUNK)) for i in range(0, N, CHUNK)]
    parts, outs = [], []
    if dout is not None:
        dout = dout.reshape(-1, N, d)
        dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    for lo, hi in spans:
        qc, kc, vc = q[:, lo:hi], k[:, lo:hi], v[:, lo:hi]
        b = g[:, lo:hi].cumsum(-1)
        D = torch.exp((b[:, :, None] - b[:, None, :]).tril()).tril()
        f, end = torch.exp(b)[..., None], torch.exp(b[:, -1:] - b)[..., None]
        pq, pk = rnd(phi(qc, kind)), rnd(phi(kc, kind))
        if dout is not None and bf16:  # the gradients take phi in two parts here
            pq = phi(qc, kind)
            P = D * (pq @ phi(kc, kind).transpose(1, 2))
        else:
            P = D * prod(pq @ pk.transpose(1, 2))
        if dout is None:
            W, Sr = rnd(P), rnd(S)
            num, den = W @ vc + f * (pq @ Sr), W.sum(-1, keepdim=True) + f * (pq @ z[..., None])
            outs.append(rnd(num / den if normalize else num))
        else:
            do = dout[:, lo:hi]
            Sr = S if bf16 else rnd(S)
            dp = prod(do @ vc.transpose(1, 2))
            Sd = f * (do @ Sr.transpose(1, 2))
            # a query's own key apart: with fast gates its weight is all but 1, and what counts is the rest
            own, val = (x.diagonal(dim1=1, dim2=2)[..., None] for x in (P, dp))
            Px, Dx = P.tril(-1), D.tril(-1)
            num = (Px * dp).sum(-1, keepdim=True) + (phi(qc, kind) * Sd).sum(-1, keepdim=True)
            den = Px.sum(-1, keepdim=True) + f * (pq @ z[..., None])
            up, delta, diff, row = torch.ones_like(num), torch.zeros_like(num), val, num
            if normalize:
                up = 1 / (den + own)
                delta = (num + own * val) * up
                diff = torch.where(own * up > 0.5, (val * den - num) * up, val - delta)
                row = -own * up * diff
            base = rnd(phi(kc, kind) - one) if kind != "relu1" or not bf16 else phi(kc, kind) - one
            X, Y = Dx * dp, Dx
            Xr = X if bf16 and one else rnd(X)
            x = Xr @ base + one * X.sum(-1, keepdim=True) + Sd
            y = rnd(Y) @ base + one * Y.sum(-1, keepdim=True) + f * z[:, None]
            dq[:, lo:hi] = rnd(up * (x - delta * y + diff * phi(kc, kind)) * slope(qc, kind))
            dgp = row[..., 0].flip(-1).cumsum(-1).flip(-1)
            parts.append((D, f, end, pq, pk, up, -delta, up * diff, dgp, S, z, b[:, -1]))
        all_ = torch.exp(b[:, -1])
        S = all_[:, None, None] * S * cross + (end * phi(kc, kind)).transpose(1, 2) @ vc
        z = all_[:, None] * z * cross + (end * phi(kc, kind)).sum(1)
        if not cross:
            S, z = S * 0, z * 0
    if dout is None:
        return torch.cat(outs, 1).reshape(*lead, N, d)
    G, h = torch.zeros_like(S), torch.zeros_like(z)
    for (lo, hi), (D, f, end, pq, pk, up, col, own, dgp, Sf, zf, last) in zip(spans[::-1], parts[::-1]):
        qc, kc, vc, do = q[:, lo:hi], k[:, lo:hi], v[:, lo:hi], dout[:, lo:hi]
        Gr, all_ = rnd(G), torch.exp(last)
        ak = end * (vc @ Gr.transpose(1, 2) + h[:, None])
        av = end * (pk @ Gr)
        W = D * up
        qk = pq @ phi(kc, kind).transpose(1, 2) if bf16 else prod(pq @ pk.transpose(1, 2))
        pw, dw = W * qk, W * (prod(do @ vc.transpose(1, 2)) + col)
        dw = dw.tril(-1) + torch.diag_embed(own[..., 0])
        base = rnd(phi(qc, kind) - one) if kind != "relu1" or not bf16 else phi(qc, kind) - one
        dv[:, lo:hi] = rnd(av + rnd(pw).transpose(1, 2) @ do)
        dk[:, lo:hi] = rnd((ak + rnd(dw).transpose(1, 2) @ base + one * dw.sum(1)[..., None]) * slope(kc, kind))
        inside = (dw * qk).tril(-1).sum(1)
        earlier = (phi(kc, kind) * ak).sum(-1)
        outside = all_ * ((Sf * G).sum((1, 2)) + (zf * h).sum(1))
        x = dgp - inside.flip(-1).cumsum(-1).flip(-1) + (earlier.cumsum(-1) - earlier) + outside[:, None]
        dg[:, lo:hi] = rnd(torch.where(g[:, lo:hi] < -104, torch.zeros_like(x), x))
        a = f * up * phi(qc, kind)
        G = cross * (all_[:, None, None] * G + a.transpose(1, 2) @ do)
        h = cross * (all_[:, None] * h + (a * col).sum(1))
    return tuple(x.reshape(*lead, *x.shape[1:]) for x in (dq, dk, dv, dg))


def norms(x, window):
    """Norms over windows of tokens of every head: [heads, windows]."""
    x = x.reshape(-1, *x.shape[2:]) if x.dim() > 2 else x
    n = x.shape[1]
    return torch.stack([x[:, i:i + window].flatten(1).norm(dim=1) for i in range(0, n, window)], 1)


def excess(got, ref, like, factor, window):
    """The largest of ||got - ref|| / (factor ||like - ref||) over heads and
    windows of tokens ([B, H, N, ...]); where `like` has no error, got must
    have none. NaN counts as infinite."""
    off, may = norms(got - ref, window), factor * norms(like - ref, window)
    r = torch.where(off <= 1e-300, torch.zeros_like(off), off / may)
    return float(torch.nan_to_num(r, nan=float("inf")).max())


def allowances(dt, *args, **kw):
    """(exact results, rounded results) of `chunked` for a type: "bf16" or "f32"."""
    rnd = to_bf16 if dt == "bf16" else fp32_noise(1)
    return chunked(*args, rnd=exact, **kw), chunked(*args, rnd=rnd, bf16=dt == "bf16", **kw)
