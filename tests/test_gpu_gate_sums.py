"""Sums of log-gates past the ends of their types: the helpers of
csrc/gate_scan.cuh through a probe (tests/cuda/gate_sums.cu), and a row of
closed gates that is longer than a sum over it could be counted."""

import ctypes
import os
import subprocess

import pytest
import torch

from kernelized_linear_attention_phi_b200 import binding as la

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe():
    from kernelized_linear_attention_phi_b200 import build
    out_dir = os.path.join(HERE, "_build")
    os.makedirs(out_dir, exist_ok=True)
    so = os.path.join(out_dir, "libgate_sums_probe.so")
    cmd = [build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", f"-I{build.CSRC}",
           f"-I{build.INCLUDE}", os.path.join(HERE, "cuda", "gate_sums.cu"), "-o", so]
    subprocess.run(cmd, check=True, capture_output=True)
    return ctypes.CDLL(so)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def pow2(probe, sums):
    b = torch.tensor(sums, dtype=torch.int64, device="cuda")
    out = torch.empty(len(sums), device="cuda")
    assert probe.gate_pow2_probe(_ptr(b), _ptr(out), len(sums)) == 0
    return out.tolist()


def test_powers_of_sums_beyond_32_bits(probe):
    inf = float("inf")
    bits = [0, -1, -126, -127, -14000, -(1 << 20), -(1 << 31), -(1 << 31) - 5, -(1 << 32) + 3, -(1 << 32),
            1, 127, 128, 14000, (1 << 31) + 5, (1 << 32) - 1]
    got = pow2(probe, [x << 31 for x in bits])
    want = [2.0 ** x if -126 <= x <= 127 else 0.0 if x < 0 else inf for x in bits]
    assert got == want


def test_sums_over_many_chunks_stop(probe):
    closed = (-14000 * 64) << 31
    b = torch.tensor([closed, closed, closed, -closed, -closed, (-3 << 31) + 5, 7 << 20], dtype=torch.int64, device="cuda")
    times = torch.tensor([1, 2397, 1 << 20, 2397, 1 << 20, 40, 1 << 10], dtype=torch.int32, device="cuda")
    total, out = torch.empty_like(b), torch.empty(len(b), device="cuda")
    assert probe.gate_add_probe(_ptr(b), _ptr(times), _ptr(total), _ptr(out), len(b)) == 0
    assert out[:3].tolist() == [0.0] * 3 and out[3:5].tolist() == [float("inf")] * 2
    assert total[5:].tolist() == [40 * ((-3 << 31) + 5), 7 << 30]
    assert (total[:5].abs() < 1 << 53).all()


def test_a_long_row_of_closed_gates():
    """One block per head, 160000 closed gates in it: the sum of their logs does not fit 32 bits in front of
    the point. Every output is its token's value, the state the last token's."""
    H, N, d = torch.cuda.get_device_properties(0).multi_processor_count, 160000, 128
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 13 GB")
    x = torch.ones(1, H, N, d, device="cuda", dtype=torch.bfloat16)
    g = torch.full((1, H, N), float("-inf"), device="cuda", dtype=torch.bfloat16)
    S, z = torch.empty(1, H, d, d, device="cuda"), torch.empty(1, H, d, device="cuda")
    out = la.la_gated_causal(x, x, x, g, S_out=S, z_out=z)
    assert bool((S == 2).all()) and bool((z == 2).all())
    assert torch.equal(out, x)


def test_a_gate_is_rounded_to_the_nearest(probe):
    """Slow gates, which a long row adds up by the thousand: no bias, and no more than half a unit each."""
    gen = torch.Generator().manual_seed(2)
    g = -torch.exp(torch.rand(1 << 16, generator=gen) * 7 - 18).cuda()  # 1.5e-8 .. 1.7e-5
    got = torch.empty(len(g), dtype=torch.int64, device="cuda")
    assert probe.gate_bits_probe(_ptr(g), _ptr(got), len(g)) == 0
    # log2 e in two doubles: the product of a 24-bit g with 29 bits of it is exact
    high = 1.44269504
    off = got.double() - (g.double() * high + g.double() * (1.4426950408889634 - high)) * 2.0 ** 31
    assert float(off.abs().max()) <= 0.5 + 2.0 ** -8
    # errors within half a unit either way: their mean over 2^16 gates is some 0.29 / 2^8
    assert abs(float(off.mean())) <= 6 * 0.29 / 2 ** 8
