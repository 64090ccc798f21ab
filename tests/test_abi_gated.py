"""Requests the gated entry points and the norm / rotation refuse, without a GPU
(validation comes before any CUDA call), and the checks of the binding."""

import ctypes

import pytest
import torch

from kernelized_linear_attention_phi_b200 import binding as B
from kernelized_linear_attention_phi_b200 import build as build_mod

P = ctypes.c_void_p(1 << 20)          # an aligned, never-dereferenced address
BAD = ctypes.c_void_p((1 << 20) + 4)  # misaligned
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def desc(B_=2, H=3, N=4000, d=64, dtype=1, phi=0, normalize=1):
    return B.la_desc(B_, H, N, d, dtype, phi, normalize)


def forward(lib, dsc, ptrs=None, ws=P, nbytes=1 << 34):
    p = dict(q=P, k=P, v=P, g=P, S_in=None, z_in=None, out=P, S_out=None, z_out=None)
    p.update(ptrs or {})
    return lib.la_gated_causal(ctypes.byref(dsc), *p.values(), ws, nbytes, None)


def backward(lib, dsc, ptrs=None, ws=P, nbytes=1 << 34):
    p = {n: P for n in ("q", "k", "v", "g", "dout", "dq", "dk", "dv", "dg")}
    p.update(ptrs or {})
    return lib.la_gated_causal_backward(ctypes.byref(dsc), *p.values(), ws, nbytes, None)


def step(lib, dsc, ptrs=None):
    p = {n: P for n in ("q", "k", "v", "g", "S", "z", "S_out", "z_out", "out")}
    p.update(ptrs or {})
    return lib.la_gated_decode_step(ctypes.byref(dsc), *p.values(), None)


def test_gated_refusals(lib):
    for call in (forward, backward, step):
        assert call(lib, desc(d=48)) == UNSUPPORTED
        assert call(lib, desc(phi=1, normalize=1)) == UNSUPPORTED
        assert call(lib, desc(B_=300, H=300)) == UNSUPPORTED
        assert call(lib, desc(B_=0)) == INVALID
        assert call(lib, desc(dtype=2)) == INVALID
        assert call(lib, desc(phi=3)) == INVALID
        for name in ("q", "g"):
            assert call(lib, desc(), {name: None}) == INVALID
            assert call(lib, desc(), {name: BAD}) == MISALIGNED
    for call in (forward, backward):
        assert call(lib, desc(N=0)) == INVALID
        assert call(lib, desc(N=-5)) == INVALID
        assert call(lib, desc(), ws=None) == WORKSPACE
        assert call(lib, desc(), nbytes=256) == WORKSPACE
        assert call(lib, desc(), ws=BAD) == MISALIGNED
    for call in (forward, backward):  # rows past 2^30 tokens
        assert call(lib, desc(B_=1, H=1, N=(1 << 30) + 1, d=16)) == UNSUPPORTED
    for one in ("S_in", "z_in", "S_out", "z_out"):
        assert forward(lib, desc(), {one: P}) == INVALID
    assert forward(lib, desc(), {"S_in": P, "z_in": BAD}) == MISALIGNED
    assert backward(lib, desc(), {"dg": None}) == INVALID
    assert backward(lib, desc(), {"dg": BAD}) == MISALIGNED
    assert step(lib, desc(), {"z_out": None}) == INVALID
    assert step(lib, desc(), {"S": BAD}) == MISALIGNED


def test_gated_workspace_sizes(lib):
    size = lambda op, **k: B.la_workspace_size(desc(**k), op)  # noqa: E731
    assert size("gated_causal") % 256 == 0 and size("gated_causal") > 0
    assert size("gated_causal", N=1) > 256 and size("gated_causal", B_=64, H=32) > 256
    assert size("gated_causal", B_=1, H=1, N=(1 << 30) + 1, d=16) == 0
    assert size("gated_causal", d=48) == 0 and size("gated_causal_bwd", N=0) == 0
    # the gradients keep a state per chunk of 64 tokens
    assert size("gated_causal_bwd") >= 2 * 3 * (-(-4000 // 64)) * (64 * 64 * 2 + 64 * 4)
    assert size("gated_causal_bwd", dtype=0) >= 2 * 3 * (4000 // 32) * (64 * 64 * 4 + 64 * 4)
    # sizes past 32 bits
    assert size("gated_causal_bwd", B_=8, H=32, N=131072, d=128) > 1 << 33


def rope_desc(**k):
    f = dict(B=2, N=100, Hq=4, Hk=2, d=64, rot=64, dtype=1, interleaved=0, table_rows=128, eps=1e-6)
    f.update(k)
    return B.la_rope_desc(*f.values())


def rope(lib, dsc, back=False, qs=(25600, 256, 64), ks=(12800, 128, 64), gs=(25600, 256, 64), nbytes=1 << 30, **k):
    p = dict(q=P, qs=None, k=P, ks=None, wq=P, wk=P, cos=P, sin=P, at=P)
    p.update({n: v for n, v in k.items() if n in p})
    s = [ctypes.byref(B.la_strides(*x)) if x else None for x in (qs, ks, gs, ks)]
    head = [ctypes.byref(dsc), p["q"], s[0], p["k"], s[1], p["wq"], p["wk"], p["cos"], p["sin"], p["at"]]
    if not back:
        return lib.la_qk_norm_rope(*head, k.get("q_out", P), k.get("k_out", P), None)
    return lib.la_qk_norm_rope_backward(*head, k.get("dyq", P), P, k.get("dq", P), s[2], P, s[3], k.get("dwq", P),
                                        k.get("dwk", P), k.get("ws", P), nbytes, None)


@pytest.mark.parametrize("back", [False, True])
def test_rope_refusals(lib, back):
    call = lambda dsc=None, **k: rope(lib, dsc or rope_desc(), back, **k)  # noqa: E731
    for bad in (dict(B=0), dict(N=-1), dict(Hq=0), dict(Hk=0), dict(dtype=7), dict(interleaved=2), dict(rot=-16),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(table_rows=0)):
        assert call(rope_desc(**bad)) == INVALID, bad
    for bad in (dict(d=96), dict(rot=80), dict(rot=24), dict(Hq=40000), dict(B=1 << 16, N=1 << 15)):
        assert call(rope_desc(**bad)) == UNSUPPORTED, bad
    assert call(rope_desc(table_rows=99), at=None) == INVALID  # positions 0 .. 99 need 100 rows
    assert call(wk=None) == INVALID and call(cos=None) == INVALID and call(qs=None) == INVALID
    assert call(q=BAD) == MISALIGNED and call(sin=BAD) == MISALIGNED
    assert call(qs=(25600, 256, 60)) == MISALIGNED
    assert call(qs=(25600, -256, 64)) == INVALID
    if back:
        assert call(gs=(25600, 0, 64)) == INVALID  # rows of a gradient on one another
        assert call(dwq=None) == INVALID and call(dq=None) == INVALID and call(dyq=BAD) == MISALIGNED
        assert call(nbytes=16) == WORKSPACE and call(ws=None) == WORKSPACE
    else:
        assert call(q_out=None) == INVALID and call(k_out=BAD) == MISALIGNED


def test_rope_workspace_size(lib):
    size = lambda **k: int(lib.la_qk_norm_rope_workspace_size(ctypes.byref(rope_desc(**k))))  # noqa: E731
    assert size() > 256 and size(d=48) == 0 and size(N=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful on a machine with no GPU")
def test_valid_requests_reach_the_device_check(lib):
    assert forward(lib, desc()) == CUDA and backward(lib, desc()) == CUDA and step(lib, desc()) == CUDA
    assert rope(lib, rope_desc()) == CUDA and rope(lib, rope_desc(), True) == CUDA
    assert rope(lib, rope_desc(rot=0, table_rows=0), cos=None, sin=None, at=None, wq=None, wk=None) == CUDA
    # strides of dimensions of size 1 are not looked at
    assert rope(lib, rope_desc(B=1, Hk=1), ks=(-3, 64, 1)) == CUDA


def test_the_binding_checks_devices_and_shapes():
    q = torch.zeros(1, 2, 8, 64)
    g = torch.zeros(1, 2, 8)
    S, z = torch.zeros(1, 2, 64, 64), torch.zeros(1, 2, 64)
    for call in (lambda: B.la_gated_causal(q, q, q, g), lambda: B.la_gated_causal_backward(q, q, q, g, q),
                 lambda: B.la_gated_decode_step(q[:, :, :1], q[:, :, :1], q[:, :, :1], g[:, :, :1], S, z),
                 lambda: B.la_qk_norm_rope(q, q, None, None, None, None),
                 lambda: B.la_qk_norm_rope_backward(q, q, None, None, None, None, q, q)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="both S and z"):
        B.la_gated_causal(q, q, q, g, S_out=S)
    with pytest.raises(ValueError, match="both S and z"):
        B.la_gated_decode_step(q[:, :, :1], q, q, g, S, z, z_out=z)
    with pytest.raises(ValueError, match="one token"):
        B.la_gated_decode_step(q, q, q, g, S, z)
    with pytest.raises(ValueError, match="B, H, N, d"):
        B.la_gated_causal(q[0], q, q, g)
    with pytest.raises(ValueError, match="dtype"):
        B.la_gated_causal(q.half(), q, q, g)
