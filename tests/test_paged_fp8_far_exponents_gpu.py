"""Attention on 8-bit rows whose values differ by many powers of two, exponents
-60 to 60: O is what the large values weigh, and L counts every key, those of
small values too, however far their share of O lies below the others'.

Checked as in test_paged_fp8_zero_values_gpu, whose tolerances count the
contributions to O and, for L, every key's rounding."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build
from test_paged_fp8_gpu import Problem, gen, status
from test_paged_fp8_zero_values_gpu import SHAPES, check, slots_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    fa2.load_library()


def problem(shape, d, below, exps_of, seed=1):
    """exps_of(n): the exponents of n keys' values.  Keys whose exponent is the largest score 0, the others -below, in
    powers of two (a query of 1 in its first element, scale 1)."""
    lens_q, lens_k, group = shape
    p = Problem(lens_q, lens_k, group, 1, d, "bf16", 16, seed=seed)
    p.q.zero_()
    p.q[..., 0] = 1.0
    g = gen(seed + 1)
    for b, n in enumerate(lens_k):
        exps = exps_of(n)
        k = torch.zeros((n, 1, d), device="cuda")
        k[:, 0, 0] = torch.where(exps == exps.max(), 0.0, -below * float(np.log(2.0)))
        # values of up to 448 * 2^e, some of them past 224
        v = (torch.rand((n, 1, d), generator=g, device="cuda", dtype=torch.float64) * 2 - 1)
        v[:, 0, 1] = 1.0
        v = v * 440 * torch.exp2(exps.double())[:, None, None]
        fa2.fa2_paged_append_fp8(k.bfloat16(), v.bfloat16(), slots_of(p, b), *p.cache)
    return p


def one_wide(at, low, high):
    def exps(n):
        e = torch.full((n,), low, device="cuda")
        e[at % n] = high
        return e
    return exps


@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("low,high", [(-60, 52), (-60, 59), (-40, 59), (-21, 59), (-20, 59), (-19, 59), (-60, 0)])
@pytest.mark.parametrize("below", [9.0, 12.0])
def test_many_small_values_beside_a_wide_one(below, low, high, shape):
    """The wide key holds nearly all of O and, beside hundreds or thousands of others, a part of the sum."""
    p = problem(SHAPES[shape], 64 if "cut" in shape else 128, below, one_wide(0, low, high))
    o, lse = p.run(window_right=0, scale=1.0)
    assert status() == fa2.FA2_OK
    check(p, o, lse, scale=1.0)


@pytest.mark.parametrize("at", [100, 127, 128, 1000, -17])
@pytest.mark.parametrize("below", [0.5, 11.0, 20.0, -3.0, -70.0])
def test_a_wide_value_behind_small_ones(at, below):
    """The sum's terms of earlier steps stay when the maximum rises by up to 120 powers of two."""
    p = problem(([1], [4000], 4), 128, below, one_wide(at, -60, 59))
    o, lse = p.run(window_right=0, scale=1.0)
    assert status() == fa2.FA2_OK
    check(p, o, lse, scale=1.0)


@pytest.mark.parametrize("n", [300, 30000])
@pytest.mark.parametrize("below", [0.0, 30.0, 75.0, -40.0])
def test_exponents_of_every_size(n, below):
    """Keys of all exponents, scores that lift the small values by what their exponents lack, or not."""
    r = gen(3)
    p = problem(([1, 2], [n, 77], 8), 128, below, lambda m: torch.randint(-60, 60, (m,), generator=r, device="cuda"))
    o, lse = p.run(window_right=0, scale=1.0)
    assert status() == fa2.FA2_OK
    check(p, o, lse, scale=1.0)


def test_zero_values_before_wide_ones():
    """Zero rows, which count with a low exponent, and behind them values of 2^68."""
    def exps(n):
        e = torch.full((n,), -8, device="cuda")
        e[200:] = 59
        return e
    p = problem(([1], [2000], 4), 128, 2.0, exps)
    zero = torch.zeros((200, 1, 128), dtype=torch.bfloat16, device="cuda")
    fa2.fa2_paged_append_fp8(zero, zero, slots_of(p, 0)[:200], *p.cache)
    o, lse = p.run(window_right=0, scale=1.0)
    assert status() == fa2.FA2_OK
    check(p, o, lse, scale=1.0)
    j = torch.arange(1800, device="cuda") % 9 == 0   # and between them
    zero = torch.zeros((int(j.sum()), 1, 128), dtype=torch.bfloat16, device="cuda")
    fa2.fa2_paged_append_fp8(zero, zero, slots_of(p, 0)[200:][j].contiguous(), *p.cache)
    o, lse = p.run(window_right=0, scale=1.0)
    assert status() == fa2.FA2_OK
    check(p, o, lse, scale=1.0)
