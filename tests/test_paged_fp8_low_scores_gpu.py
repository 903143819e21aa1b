"""Attention on 8-bit rows at scores far from zero: `scale` may be any finite
value, and a key counts as long as its score is a finite fp32 number.

Scores here are equal for all keys, or some of them far below the others, so
that the weights are exact: 1 / n each, or 0.  All values have size 0.5, with
one exponent.  Tolerances: O is rounded once (u = eps / 2) from n terms added in
fp32 and P of 12 bits, (2^-12 + 2 n 2^-23) A with A = 0.5; L is a sum of n equal
terms (n 2^-23 and 2^-18, as test_paged_fp8_gpu) and a score of a product of
five factors in fp32, 2^-22 |L|."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build
from test_paged_fp8_gpu import DT, Problem, gen, status
from test_paged_fp8_zero_values_gpu import SHAPES, slots_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    fa2.load_library()


def problem(shape, d, dtype, key_of):
    """Queries of 1 in their first element; key j of sequence b has key_of(b, n)[j] there."""
    lens_q, lens_k, group = shape
    p = Problem(lens_q, lens_k, group, 1, d, dtype, 16, seed=1)
    p.q.zero_()
    p.q[..., 0] = 1.0
    p.values = []
    for b, n in enumerate(lens_k):
        k = torch.zeros((n, 1, d), device="cuda")
        k[:, 0, 0] = key_of(b, n)
        v = torch.randint(0, 2, (n, 1, d), generator=gen(b), device="cuda") - 0.5
        p.values.append(v[:, 0].double())
        if n:
            fa2.fa2_paged_append_fp8(k.to(DT[dtype]), v.to(DT[dtype]), slots_of(p, b), *p.cache)
    return p


def check(p, o, lse, score, weigh):
    """Every row has the keys that weigh(b, n) marks among those it sees, of one score each."""
    u, row = torch.finfo(o.dtype).eps / 2, 0
    for b, (n_q, n) in enumerate(zip(p.lens_q, p.lens_k)):
        for i in range(n_q):
            got_o, got_l = o[row + i].double(), lse[:, row + i].double()
            end = n - n_q + i + 1
            marked = weigh(b, n)[:max(end, 0)]
            count = int(marked.sum())
            if count == 0:
                assert (got_o == 0).all() and torch.isneginf(got_l).all()
                continue
            ref = p.values[b][:end][marked].mean(0)
            tol = u * ref.abs() + 0.5 * (2.0 ** -12 + 2 * count * 2.0 ** -23)
            assert torch.isfinite(got_o).all() and ((got_o - ref).abs() <= tol).all(), (b, i)
            ref_l = score + np.log(count)
            assert ((got_l - ref_l).abs() <= count * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22 * abs(ref_l)).all(), (b, i)
        row += n_q


@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("scale,key", [(1e30, -2.0), (-1e30, 2.0), (1e38, -2.0), (1e38, 2.0), (6e29, -1.0), (1.0, -240.0)])
def test_equal_scores(scale, key, shape):
    p = problem(SHAPES[shape], 64 if "cut" in shape else 128, "bf16", lambda b, n: torch.full((n,), key, device="cuda"))
    o, lse = p.run(window_right=0, scale=scale)
    assert status() == fa2.FA2_OK
    check(p, o, lse, scale * key, lambda b, n: torch.ones(n, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", ["8", "8 cut", "16", "32"])
@pytest.mark.parametrize("scale,low,high", [(1e30, -4.0, -2.0), (1e38, -2.0, -1.0), (1e38, -2.0, 2.0), (1e30, -2.0, 0.0)])
def test_later_keys_far_above_the_first(scale, low, high, shape, dtype):
    """The last key of every 200, and from one step of 128 keys on: all weight is theirs."""
    at = lambda b, n: torch.arange(n, device="cuda") % 200 == min(199, n // 2)
    p = problem(SHAPES[shape], 128, dtype, lambda b, n: torch.where(at(b, n), high, low))
    o, lse = p.run(scale=scale)
    assert status() == fa2.FA2_OK
    p.lens_q = [1] * len(p.lens_q)   # without a causal edge every row is the last one's
    last = np.cumsum(SHAPES[shape][0]) - 1
    check(p, o[last], lse[:, last], scale * high, at)


def test_rows_without_keys_beside_low_scores():
    p = problem(([5, 1, 3], [3, 0, 40], 4), 128, "bf16", lambda b, n: torch.full((n,), -2.0, device="cuda"))
    o, lse = p.run(window_right=0, scale=1e30)
    assert status() == fa2.FA2_OK
    check(p, o, lse, -2e30, lambda b, n: torch.ones(n, dtype=torch.bool, device="cuda"))


def test_as_the_16_bit_forward_on_the_rows_read_back():
    p = problem(([1, 3], [300, 40], 4), 128, "bf16", lambda b, n: torch.full((n,), -2.0, device="cuda"))
    o, lse = p.run(window_right=0, scale=1e30)
    pages = p.cache[0].shape[0]
    k, v = fa2.fa2_paged_read_fp8(torch.arange(pages * 16, dtype=torch.int32, device="cuda"), *p.cache)
    k16, v16 = (x.view(pages, 16, 1, 128).transpose(1, 2) for x in (k, v))
    o16, lse16 = fa2.fa2_paged_fwd(p.q, k16, v16, p.table, p.cu, p.lens, window_right=0, max_seqlen_q=3, scale=1e30)
    assert status() == fa2.FA2_OK
    assert torch.allclose(lse, lse16, rtol=2.0 ** -21, atol=0)
    assert (o.float() - o16.float()).abs().max() <= 2 * 2.0 ** -8 * 0.5
