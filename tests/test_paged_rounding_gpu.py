"""Where the paged forward keeps the low part of bf16 P: on the key tiles that the
mask cuts and where a sequence has few keys, whichever kernel the batch gets.

Queries and keys are small integers, so every score is exact in fp32, and the
weight of a row lies on keys of cut tiles.  Per element, with A = sum p |v|, u =
2^-8 and x the largest |score| times log2 e among the keys that weigh:
- P = P_hi + P_lo is off by at most u^2 = 2^-16 of each term;
- the exponent's scale and its one FMA are off by 2^-24 of x each, and the
  exponential by 2^-22: twice that much of A, for P and for their sum;
- sums of n terms in fp32, the merge and the division: (2 n 2^-23 + 2^-18) A;
- O is rounded once: u |O|;
- the keys outside cut tiles weigh w in all: u w max |v|.
One rounded P alone would be off by up to u A, 2^8 times the first term."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build
from test_paged_gpu import Problem, seen_mask, status

pytestmark = pytest.mark.gpu

SCALE = 0.1


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    fa2.load_library()


def integers(p, heavy, seed):
    """q and k in -1 .. 1; the first two columns add 25.6 to the scores of each sequence's heavy keys."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for x in (p.q, p.k):
        x.copy_(torch.randint(-1, 2, x.shape, generator=g, device="cuda").to(x.dtype))
    p.q[..., :2] = 8
    for b, (lo, hi) in enumerate(heavy):
        j = torch.arange(lo, hi, device="cuda")
        p.k[p.table[b, j // p.page].long(), :, j % p.page, :2] = 16


def check(p, o, heavy, wl):
    u, row = 2.0 ** -8, 0
    for b, (n, n_k) in enumerate(zip(p.lens_q, p.lens_k)):
        j = torch.arange(n_k, device="cuda")
        pg = p.table[b, j // p.page].long()
        rep = p.hq // p.hkv
        k, v = (c[pg, :, j % p.page].double().transpose(0, 1).repeat_interleave(rep, 0) for c in (p.k, p.v))
        s = SCALE * (p.q[row:row + n].double().transpose(0, 1) @ k.transpose(1, 2))
        s = s.masked_fill(~seen_mask(n, n_k, wl, 0, 0), -np.inf)
        w = torch.softmax(s, -1)
        want, a = w @ v, w @ v.abs()
        out = (j < heavy[b][0]) | (j >= heavy[b][1])
        w_out = w[..., out].sum(-1)
        assert w_out.max() < 1e-6
        x = (s[..., ~out].masked_fill(torch.isinf(s[..., ~out]), 0).abs().amax(-1) * 1.4427)[..., None]
        tol = u * want.abs() + u * w_out[..., None] * v.abs().max() + 1e-7
        tol += a * (2.0 ** -16 + 2 * (2 * x * 2.0 ** -24 + 2.0 ** -22) + 2 * n_k * 2.0 ** -23 + 2.0 ** -18)
        worst = ((o[row:row + n].double().transpose(0, 1) - want).abs() / tol).max()
        assert worst <= 1, "sequence %d: off by %.2f tolerances" % (b, worst)
        row += n


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("max_q", [20, 128])   # query tiles of few rows and of many
@pytest.mark.parametrize("edge", ["right", "left", "few"])
def test_low_part_of_p_on_cut_tiles(edge, max_q, d):
    lens_q = [1, 5, 1, 16, 3, 1]
    if edge == "right":     # all rows end in the last, partial tile
        lens_k = [64 * t + 37 for t in (5, 9, 140, 4, 30, 7)]
        heavy, wl = [(n // 64 * 64, n) for n in lens_k], -1
    elif edge == "left":    # all rows' windows of 300 start in one tile
        lens_k = [64 * t + 44 + 20 + q for t, q in zip((8, 9, 40, 11, 30, 7), lens_q)]
        heavy, wl = [(n - 301, (n - 301) // 64 * 64 + 64) for n in lens_k], 300
    else:                   # all keys in three tiles
        lens_k, wl = [192, 100, 65, 150, 64, 127], -1
        heavy = [(0, n) for n in lens_k]
    p = Problem(lens_q, lens_k, 6, 2, d, "bf16", 16, seed=d)
    integers(p, heavy, seed=d + 1)
    o, _ = p.run(window_left=wl, window_right=0, scale=SCALE, max_seqlen_q=max_q)
    assert status() == fa2.FA2_OK
    check(p, o, heavy, wl)
