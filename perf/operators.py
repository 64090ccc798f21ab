"""Cases of the gated linear attention and of the query / key preparation, with
their plain forms.

``kind`` names the operator:

* ``gated``: la_gated_causal, the causal form of S_t = exp(g_t) S_{t-1} + phi(k_t) v_t,
  with the state after the last token (and, with ``start``, a state to begin from);
* ``gated_bwd``: la_gated_causal_backward, the gradients of q, k, v and g;
* ``gated_step``: la_gated_decode_step, one token on a cached state;
* ``rope``: la_qk_norm_rope, the norm of every query and key row with the
  position rotation, out of a packed projection into [B, H, N, d];
* ``rope_bwd``: la_qk_norm_rope_backward.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-6
CHUNK = 64
CLOSED = -1e4  # log-gate that stands for -inf in the plain form's sums


def _gated(name, kind, B, H, N, d, dtype, phi, normalize, **more):
    c = {"name": name, "kind": kind, "B": B, "H": H, "N": N, "d": d, "dtype": dtype, "phi": phi,
         "normalize": normalize, "start": False, "docs": 0}
    c.update(more)
    return c


def _rope(name, kind, B, N, Hq, Hk, d, dtype, rot, interleaved, positions):
    return {"name": name, "kind": kind, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "d": d, "dtype": dtype, "rot": rot,
            "interleaved": interleaved, "positions": positions}


def listed():
    return [
        # prompt of the multi-head layer (2 x 4096 tokens, 8 heads of 64)
        _gated("prefill", "gated", 2, 8, 4096, 64, "bf16", "relu1", True),
        # one long context, the largest call: few heads, so the time axis is split
        _gated("prefill_long", "gated", 1, 16, 131072, 128, "bf16", "relu1", True),
        # a later piece of a prompt in full precision, odd length, from a cached state, with documents packed into the rows
        _gated("prefill_piece_f32", "gated", 1, 4, 1531, 32, "f32", "elu1", True, start=True, docs=3),
        # the training step of the multi-head layer
        _gated("train", "gated_bwd", 2, 8, 4096, 64, "bf16", "relu1", True),
        # a long training row of packed documents, unnormalized identity map
        _gated("train_long", "gated_bwd", 1, 16, 32768, 128, "bf16", "identity", False, docs=9),
        # a full-precision step with a ragged length
        _gated("train_f32", "gated_bwd", 2, 4, 1000, 64, "f32", "relu1", True),
        # a full decode batch: 64 sequences, 32 heads of 128
        _gated("step", "gated_step", 64, 32, 1, 128, "bf16", "relu1", True),
        # one sequence alone: latency
        _gated("step_single", "gated_step", 1, 8, 1, 64, "bf16", "relu1", True),
        # long prompts of the 16-head layer, half-split rotation of the whole head
        _rope("rope_prefill", "rope", 4, 16384, 16, 16, 64, "bf16", 64, False, "rows"),
        # one token of each of 64 sequences, each at its own position
        _rope("rope_step", "rope", 64, 1, 32, 32, 128, "bf16", 128, False, "any"),
        # the training step of the multi-head layer, interleaved rotation
        _rope("rope_train", "rope_bwd", 2, 4096, 8, 8, 64, "bf16", 64, True, "rows"),
        # full precision, odd length, fewer key heads, a partly rotated head
        _rope("rope_train_f32", "rope_bwd", 3, 1777, 12, 4, 128, "f32", 64, False, "any"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gated", "gated", "gated_bwd", "gated_bwd", "gated_step", "rope", "rope_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([16, 32, 64, 64, 128, 128])
    if kind.startswith("gated"):
        phi, normalize = rng.choice([("relu1", True), ("relu1", False), ("elu1", True), ("identity", False)])
        c = {"kind": kind, "B": _log(rng, 1, 8), "H": _log(rng, 1, 32), "N": 1, "d": d, "dtype": dtype, "phi": phi,
             "normalize": normalize, "start": False, "docs": 0}
        if kind == "gated_step":
            c["B"] = _log(rng, 1, 64)
        else:
            # at most 2^24 elements of q in a gradient, 2^26 in a forward call
            most = (1 << (24 if kind == "gated_bwd" else 26)) // (c["B"] * c["H"] * d)
            # a normalized gradient of one token is exactly zero: nothing to compare
            c["N"] = _log(rng, 8 if kind == "gated_bwd" else 1, max(8, min(most, 4096 if dtype == "f32" else 65536)))
            c["start"] = kind == "gated" and rng.random() < 0.4
            c["docs"] = rng.choice([0, 0, 2, 5])
        return c
    B, Hk = _log(rng, 1, 64), _log(rng, 1, 16)
    Hq = Hk * rng.choice([1, 1, 2, 4])
    most = (1 << 26) // (B * Hq * d)
    return {"kind": kind, "B": B, "N": _log(rng, 1, max(2, min(most, 32768))), "Hq": Hq, "Hk": Hk, "d": d, "dtype": dtype,
            "rot": rng.choice([d, d, max(16, d // 2)]), "interleaved": rng.random() < 0.5, "positions": rng.choice(["rows", "any"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1_000_003 * int(seed) + 17)
    dt = DT[case["dtype"]]

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * sigma

    s = dict(case)
    d, B = case["d"], case["B"]
    if case["kind"].startswith("gated"):
        H, N = case["H"], case["N"]
        sigma = 1.0 if case["phi"] != "identity" else d ** -0.5
        s["q"], s["k"], s["v"] = (normal(B, H, N, d, sigma=sigma).to(dt) for _ in range(3))
        # heads remember from some tokens to some thousand; each token scales its head's decay
        span = torch.exp(torch.rand(H, generator=gen, device="cuda") * math.log(512.0)) * 4.0
        g = -torch.exp(0.5 * normal(B, H, N)) / span.view(1, H, 1)
        if case["docs"] and N > 1:  # a document starts where the gate is closed
            at = torch.randint(1, N, (B, case["docs"]), generator=gen, device="cuda")
            g.scatter_(2, at[:, None, :].expand(B, H, case["docs"]), float("-inf"))
        s["g"] = g.to(dt)
        if case["start"] or case["kind"] == "gated_step":
            # the state of a prompt: a sum of outer products of some hundred tokens
            kk, vv = normal(B, H, 256, d, sigma=sigma), normal(B, H, 256, d, sigma=sigma)
            kk = _phi(kk, case["phi"])
            s["S"], s["z"] = (kk.transpose(2, 3) @ vv).contiguous(), kk.sum(2).contiguous()
        if case["kind"] == "gated_bwd":
            s["dout"] = normal(B, H, N, d).to(dt)
        return s
    N, Hq, Hk, rot = case["N"], case["Hq"], case["Hk"], case["rot"]
    packed = normal(B, N, (Hq + 2 * Hk) * d).to(dt)
    s["packed"] = packed
    s["q"] = packed[..., :Hq * d].view(B, N, Hq, d)
    s["k"] = packed[..., Hq * d:(Hq + Hk) * d].view(B, N, Hk, d)
    s["wq"], s["wk"] = 1.0 + 0.1 * normal(d), 1.0 + 0.1 * normal(d)
    rows = max(N, 4096)
    freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["at"] = None
    if case["positions"] == "any":
        s["at"] = torch.randint(0, rows, (B, N), generator=gen, device="cuda", dtype=torch.int32)
    if case["kind"] == "rope_bwd":
        s["dq"], s["dk"] = normal(B, Hq, N, d).to(dt), normal(B, Hk, N, d).to(dt)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _phi(x, phi):
    if phi == "relu1":
        return torch.where(x > 0, x, torch.zeros_like(x)) + 1
    if phi == "elu1":
        return torch.where(x > 0, x + 1, torch.exp(torch.minimum(x, torch.zeros_like(x))))
    return x


def _decay(upto, frm, keep):
    """exp(upto - frm) where `keep`, else 0, of 64-bit sums."""
    zero = torch.zeros((), dtype=torch.float64, device=upto.device)
    return torch.where(keep, torch.exp(torch.where(keep, upto - frm, zero)), zero).float()


def _plain_gated(q, k, v, g, phi, normalize, S0=None, z0=None):
    """Chunks of 64 tokens: products inside a chunk under its decay matrix, and
    the states of the earlier chunks under the decay matrix of the chunks."""
    B, H, N, d = q.shape
    a, b, v = _phi(q.float(), phi), _phi(k.float(), phi), v.float()
    v = torch.cat([v, torch.ones_like(v[..., :1])], -1)
    n = -(-N // CHUNK)
    pad = n * CHUNK - N
    a, b, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, n, CHUNK, -1) for x in (a, b, v))
    logs = torch.nn.functional.pad(g.double().clamp(min=CLOSED), (0, pad)).view(B, H, n, CHUNK).cumsum(-1)
    total = logs[..., -1].cumsum(-1)                                  # up to the end of each chunk
    before = total - logs[..., -1]                                    # up to its start
    idx = torch.arange(CHUNK, device=q.device)
    inner = _decay(logs[..., :, None], logs[..., None, :], idx[:, None] >= idx[None, :])
    own_kv = (b * torch.exp(logs[..., -1:] - logs).float()[..., None]).transpose(-1, -2) @ v   # [B, H, n, d, d + 1]
    chunk = torch.arange(n, device=q.device)
    outer = _decay(before[..., :, None], total[..., None, :], chunk[:, None] > chunk[None, :])
    start = (outer @ own_kv.reshape(B, H, n, -1)).view(B, H, n, d, d + 1)
    if S0 is not None:
        first = torch.cat([S0, z0[..., None]], -1)
        start = start + torch.exp(before).float()[..., None, None] * first[:, :, None]
    num = ((a @ b.transpose(-1, -2)) * inner) @ v + torch.exp(logs).float()[..., None] * (a @ start)
    end = torch.exp(logs[..., -1, -1]).float()[..., None, None] * start[:, :, -1] + own_kv[:, :, -1]
    num = num.reshape(B, H, n * CHUNK, d + 1)[:, :, :N]
    out = num[..., :d] / num[..., d:] if normalize else num[..., :d]
    return out, end[..., :d].contiguous(), end[..., d].contiguous()


def _plain_gated_backward(s):
    q, k, v, g = (s[x].float().requires_grad_() for x in "qkvg")
    with torch.enable_grad():
        out, _, _ = _plain_gated(q, k, v, g, s["phi"], s["normalize"])
        grads = torch.autograd.grad(out, (q, k, v, g), s["dout"].float())
    return tuple(x.to(s["q"].dtype) for x in grads)


def _plain_step(s):
    q, k, v = (s[x][:, :, 0].float() for x in "qkv")
    a, b = _phi(q, s["phi"]), _phi(k, s["phi"])
    decay = torch.exp(s["g"][:, :, 0].float())
    S = decay[..., None, None] * s["S"] + b[..., :, None] * v[..., None, :]
    z = decay[..., None] * s["z"] + b
    out = (a[..., None] * S).sum(-2)
    if s["normalize"]:
        out = out / (a * z).sum(-1, keepdim=True)
    return out[:, :, None].to(s["q"].dtype), S, z


def _turn(x, cos, sin, interleaved, back):
    """The rotation of the first 2 * len(cos) channels; `back` turns the other way."""
    half = cos.shape[-1]
    first, second = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    if back:
        sin = -sin
    one, two = first * cos - second * sin, second * cos + first * sin
    turned = torch.stack([one, two], -1).flatten(-2) if interleaved else torch.cat([one, two], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _angles(s):
    B, N = s["B"], s["N"]
    if s["at"] is None:
        return s["cos"][None, :N, None], s["sin"][None, :N, None]
    at = s["at"].long().view(-1)
    return (s[t][at].view(B, N, 1, -1) for t in ("cos", "sin"))


def _plain_rope(s):
    cos, sin = _angles(s)
    outs = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.float()
        u = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
        outs.append(_turn(u, cos, sin, s["interleaved"], False).transpose(1, 2).to(x.dtype).contiguous())
    return tuple(outs)


def _plain_rope_backward(s):
    cos, sin = _angles(s)
    grads, weights = [], []
    for x, w, dy in ((s["q"], s["wq"], s["dq"]), (s["k"], s["wk"], s["dk"])):
        y = x.float()
        r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
        n = y * r
        du = _turn(dy.float().transpose(1, 2), cos, sin, s["interleaved"], True)
        dn = du * w
        grads.append((r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype))
        weights.append((du * n).sum((0, 1, 2), dtype=torch.float64).float())
    return (*grads, *weights)


def run(state):
    s = state
    kind = s["kind"]
    if own:
        from kernelized_linear_attention_phi_b200 import binding as la

        how = {"phi": s.get("phi"), "normalize": s.get("normalize")}
        if kind == "gated":
            B, H, _, d = s["q"].shape
            S = torch.empty(B, H, d, d, device="cuda")
            z = torch.empty(B, H, d, device="cuda")
            out = la.la_gated_causal(s["q"], s["k"], s["v"], s["g"], S_in=s.get("S"), z_in=s.get("z"), S_out=S, z_out=z, **how)
            return out, S, z
        if kind == "gated_bwd":
            return la.la_gated_causal_backward(s["q"], s["k"], s["v"], s["g"], s["dout"], **how)
        if kind == "gated_step":
            S, z = torch.empty_like(s["S"]), torch.empty_like(s["z"])
            out = la.la_gated_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], s["z"], S_out=S, z_out=z, **how)
            return out, S, z
        how = {"positions": s["at"], "eps": EPS, "interleaved": s["interleaved"]}
        if kind == "rope":
            return la.la_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], **how)
        return la.la_qk_norm_rope_backward(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["dq"], s["dk"], **how)
    if kind == "gated":
        out, S, z = _plain_gated(s["q"], s["k"], s["v"], s["g"], s["phi"], s["normalize"], s.get("S"), s.get("z"))
        return out.to(s["q"].dtype), S, z
    if kind == "gated_bwd":
        return _plain_gated_backward(s)
    if kind == "gated_step":
        return _plain_step(s)
    return _plain_rope(s) if kind == "rope" else _plain_rope_backward(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    e, d, B = SIZE[case["dtype"]], case["d"], case["B"]
    if case["kind"].startswith("gated"):
        rows = B * case["H"] * case["N"]
        state = B * case["H"] * (d * d + d) * 4
        if case["kind"] == "gated_step":
            return {"bytes": 2 * state + rows * (4 * d + 1) * e, "flops": rows * 5 * d * d}
        if case["kind"] == "gated":  # per token: the state's update and the readout, both d x d
            return {"bytes": rows * (4 * d + 1) * e + state * (2 if case["start"] else 1), "flops": rows * 5 * d * d}
        return {"bytes": rows * (7 * d + 2) * e, "flops": rows * 12 * d * d}
    rows = B * case["N"] * (case["Hq"] + case["Hk"])
    seen = B * case["N"] if case["positions"] == "any" else case["N"]
    small = min(seen, max(case["N"], 4096)) * case["rot"] * 4 + (B * case["N"] * 4 if case["positions"] == "any" else 0)
    if case["kind"] == "rope":
        return {"bytes": rows * 2 * d * e + small + 2 * d * 4, "flops": rows * 8 * d}
    return {"bytes": rows * 3 * d * e + small + 4 * d * 4, "flops": rows * 14 * d}


def _exact_gated(s):
    """The recurrence itself, token by token, in 64 bits."""
    B, H, N, d = s["q"].shape
    q, k, v, g = (s[x].double() for x in "qkvg")
    a, b, decay = _phi(q, s["phi"]), _phi(k, s["phi"]), torch.exp(g)
    v1 = torch.cat([v, torch.ones_like(v[..., :1])], -1)
    S = torch.zeros(B, H, d, d + 1, dtype=torch.float64, device=q.device)
    if "S" in s:
        S = torch.cat([s["S"].double(), s["z"].double()[..., None]], -1)
    back = s["kind"] == "gated_bwd"
    num = torch.empty_like(v1)
    da = torch.empty_like(q)
    if back:
        dout, ups = s["dout"].double(), torch.empty_like(v1)
    for t in range(N):
        S = S * decay[:, :, t, None, None] + b[:, :, t, :, None] * v1[:, :, t, None, :]
        num[:, :, t] = (a[:, :, t, None, :] @ S)[:, :, 0]
        if back:
            up = dout[:, :, t]
            if s["normalize"]:
                up = up / num[:, :, t, d:]
                up = torch.cat([up, -(up * num[:, :, t, :d]).sum(-1, keepdim=True) / num[:, :, t, d:]], -1)
            else:
                up = torch.cat([up, torch.zeros_like(up[..., :1])], -1)
            da[:, :, t] = (S @ up[..., None])[..., 0]
            ups[:, :, t] = up
    if not back:
        out = num[..., :d] / num[..., d:] if s["normalize"] else num[..., :d]
        return out, S[..., :d], S[..., d]
    G = torch.zeros_like(S)
    db, dv = torch.empty_like(q), torch.empty_like(q)
    for t in range(N - 1, -1, -1):
        G = G + a[:, :, t, :, None] * ups[:, :, t, None, :]
        db[:, :, t] = (G @ v1[:, :, t, :, None])[..., 0]
        dv[:, :, t] = (b[:, :, t, None, :] @ G)[:, :, 0, :d]
        G = G * decay[:, :, t, None, None]

    def slope(x):
        if s["phi"] == "identity":
            return torch.ones_like(x)
        return torch.where(x > 0, torch.ones_like(x), torch.zeros_like(x) if s["phi"] == "relu1" else torch.exp(x))

    # <S_t, G_t> = dg_t + b_t . db_t = a_t . da_t + dg_{t + 1}
    dg = ((a * da).sum(-1) - (b * db).sum(-1)).flip(-1).cumsum(-1).flip(-1)
    return da * slope(q), db * slope(k), dv, torch.where(decay > 0, dg, torch.zeros_like(dg))


def _exact_rope(s):
    at = s["at"].long() if s["at"] is not None else torch.arange(s["N"], device="cuda").expand(s["B"], s["N"])
    cos, sin = s["cos"].double()[at][:, :, None], s["sin"].double()[at][:, :, None]
    half, d = s["rot"] // 2, s["d"]
    i = torch.arange(half, device="cuda")
    one, two = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    outs, weights = [], []
    for x, w, dy in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double(), w.double()
        r = (x.square().sum(-1, keepdim=True) / d + EPS) ** -0.5
        if dy is None:
            y = x * r * w
            u = y.clone()
            y[..., one] = cos * u[..., one] - sin * u[..., two]
            y[..., two] = sin * u[..., one] + cos * u[..., two]
            outs.append(y.transpose(1, 2))
            continue
        dy = dy.double().transpose(1, 2)
        du = dy.clone()
        du[..., one] = cos * dy[..., one] + sin * dy[..., two]
        du[..., two] = cos * dy[..., two] - sin * dy[..., one]
        weights.append((du * x * r).sum((0, 1, 2)))
        du = du * w
        outs.append(r * du - x * r ** 3 * (du * x).sum(-1, keepdim=True) / d)
    return (*outs, *weights)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"].startswith("gated"):
        return _exact_gated(s)
    return _exact_rope(s)
