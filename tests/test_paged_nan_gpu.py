"""NaN in what a row of the paged forward sees reaches that row's O and LSE, and
no row that does not see it: a corrupt page must not pass for a row without keys
(O = 0, LSE = -inf)."""
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build
from test_paged_gpu import Problem, status

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    fa2.load_library()


def expect_nan(got, clean, hit):
    """O and LSE are NaN in the rows hit ([total_q, H]) and unchanged in the others."""
    (o, lse), (o0, lse0) = got, clean
    assert status() == fa2.FA2_OK
    assert o[hit].isnan().all() and lse.t()[hit].isnan().all()
    assert torch.equal(o[~hit], o0[~hit]) and torch.equal(lse.t()[~hit], lse0.t()[~hit])


# whole pairs (short), pairs cut over many CTAs (long), few and many rows
SHAPES = {"short": ([1, 3], [40, 100]), "long": ([1, 2], [9000, 5000]), "chunk": ([70, 1], [70, 300]),
          "long chunk": ([200], [9000]), "many": ([1] * 40, [1000 + 9 * b for b in range(40)])}


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (128, "fp16"), (256, "fp16")])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_nan_in_a_query(shape, d, dtype):
    lens_q, lens_k = SHAPES[shape]
    p = Problem(lens_q, lens_k, 8, 2, d, dtype, 16, seed=d)
    clean = p.run(window_right=0)
    hit = torch.zeros(p.q.shape[:2], dtype=torch.bool, device="cuda")
    for row, head in ((0, 1), (sum(lens_q) - 1, 7)):
        p.q[row, head, row % d] = NAN
        hit[row, head] = True
    expect_nan(p.run(window_right=0), clean, hit)


@pytest.mark.parametrize("mask", [dict(window_right=0), dict(window_left=500, window_right=0, prefix_len=4)])
@pytest.mark.parametrize("at", ["first", "middle", "last", "all"])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_nan_in_keys(shape, at, mask):
    """Keys of the last sequence and of one K/V head: the rows that see one of them, in that head's group."""
    lens_q, lens_k = SHAPES[shape]
    p = Problem(lens_q, lens_k, 8, 2, 128, "bf16", 16, seed=3)
    clean = p.run(**mask)
    b, n_k, n = len(lens_k) - 1, lens_k[-1], lens_q[-1]
    keys = {"first": [0], "middle": [n_k // 2], "last": [n_k - 1], "all": range(n_k)}[at]
    j = torch.tensor(list(keys), device="cuda")
    p.k[p.table[b, j // 16].long(), 1, j % 16, 5] = NAN
    i = torch.arange(n_k - n, n_k, device="cuda")[:, None]
    sees = (j <= i) & ((j >= i - 500) | (j < 4) if "window_left" in mask else True) | (j < mask.get("prefix_len", 0))
    hit = torch.zeros(p.q.shape[:2], dtype=torch.bool, device="cuda")
    hit[-n:, 4:] = sees.any(1)[:, None]
    expect_nan(p.run(**mask), clean, hit)


def test_nan_in_a_value():
    """Every row of a decoding batch that sees it, in that column of that head's group; the scores do not."""
    p = Problem([1, 1], [3000, 50], 8, 2, 128, "bf16", 16, seed=4)
    o0, lse0 = p.run(window_right=0)
    p.v[p.table[0, 7].long(), 0, 3, 9] = NAN
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK and torch.equal(lse, lse0)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[0, :4, 9] = True
    assert o[hit].isnan().all() and torch.equal(o[~hit], o0[~hit])
