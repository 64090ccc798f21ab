"""Strides of the gradients that la_qk_norm_rope_backward writes: rows that fall
on one another are refused, every other view is taken (validation comes before
any CUDA call; no GPU)."""

import ctypes
import itertools
import random

import pytest
import torch

from kernelized_linear_attention_phi_b200 import binding as B
from kernelized_linear_attention_phi_b200 import build as build_mod

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="valid requests are launched where there is a GPU")

P = ctypes.c_void_p(1 << 20)  # an aligned, never-dereferenced address
INVALID, CUDA = 1, 5


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


def backward(lib, sizes, strides, d=16):
    """Status for dq of [B, N, H, d] with these strides (q and dk contiguous)."""
    b, n, h = sizes
    desc = B.la_rope_desc(b, n, h, 1, d, 0, 1, 0, 0, 1e-6)
    s = [ctypes.byref(B.la_strides(*x)) for x in ((n * h * d, h * d, d), (n * d, d, d), strides)]
    return lib.la_qk_norm_rope_backward(ctypes.byref(desc), P, s[0], P, s[1], None, None, None, None, None, P, P, P, s[2],
                                        P, s[1], None, None, P, 1 << 40, None)


def overlap(sizes, strides, d):
    starts = sorted(sum(i * s for i, s in zip(at, strides)) for at in itertools.product(*map(range, sizes)))
    return any(b - a < d for a, b in zip(starts, starts[1:]))


def test_rows_on_one_another_are_refused(lib):
    assert backward(lib, (2, 3, 4), (192, 16, 16)) == INVALID      # tokens and heads step alike
    assert backward(lib, (2, 3, 4), (64, 64, 16)) == INVALID       # sequences and tokens
    assert backward(lib, (2, 3, 4), (192, 64, 24)) == INVALID      # the next token starts inside the last head
    assert backward(lib, (2, 1 << 20, 2), (16, 16, 1 << 30)) == INVALID


def test_against_a_search_over_all_rows(lib):
    rng = random.Random(3)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        sizes = tuple(rng.choice([1, 2, 3, 5]) for _ in range(3))
        strides = tuple(8 * rng.choice([2, 2, 3, 4, 5, 6, 9, 12, 20, 33]) for _ in range(3))
        bad = overlap([n for n in sizes], [0 if n == 1 else s for n, s in zip(sizes, strides)], 16)
        assert backward(lib, sizes, strides) == (INVALID if bad else CUDA), (sizes, strides)
        seen[bad] += 1
    assert min(seen.values()) > 500
    assert backward(lib, (1, 1 << 30, 1), (1, 24, 1)) == CUDA
    # the packed and the permuted views of a projection's gradient
    for strides in ((640, 160, 16), (640, 16, 160), (160, 640, 16), (16, 128, 640)):
        assert backward(lib, (4, 4, 3), strides) == CUDA, strides
