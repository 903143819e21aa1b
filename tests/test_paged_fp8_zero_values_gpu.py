"""Attention on 8-bit rows where value rows are zero and carry weight: a null or
sink key, padding that a prompt holds, a page out of range (which reads as zero
codes).  Such a key adds to the row's sum and nothing to O, so it must take no
precision from the others' share of O.

The tolerance of O counts roundings as test_paged_fp8_gpu does (u = eps / 2 of
the 16-bit type, A = sum p |v|), but for the third part of P, whose smallest
step rounds by 2^-18 where the row's largest P 2^e is at least 2^4: 2^-22 of the
largest p 2^e for every key's |code|, and only over the keys that add to O.  A
row's largest code is 224 or more unless its exponent is at its lower end, so
that p 2^e is p max |v| / 224 at most, or p times the lowest power of two."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build
from test_paged_fp8_gpu import DT, LIMITS, Problem, gen, seen_mask, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    fa2.load_library()


def slots_of(p, b):
    j = torch.arange(p.lens_k[b], device="cuda")
    return (p.table[b, j // p.page].long() * p.page + j % p.page).to(torch.int32)


def check(p, o, lse, scale=None, window_left=-1, window_right=0, prefix_len=0, sink_len=0):
    group = p.hq // p.hkv
    scale = 1.0 / p.d ** 0.5 if scale is None else scale
    u, least = torch.finfo(o.dtype).eps / 2, 2.0 ** LIMITS[o.dtype][0]
    denormal = 2.0 ** -25 if o.dtype == torch.float16 else 0.0   # half of fp16's smallest step
    row = 0
    for b, (n, n_k) in enumerate(zip(p.lens_q, p.lens_k)):
        (kc, ke), (vc, ve) = p.keys(b, 0), p.keys(b, 1)
        k, v, vc, ve = (x.repeat_interleave(group, 0) for x in (
            kc * torch.exp2(ke)[..., None], vc * torch.exp2(ve)[..., None], vc, ve))
        hidden = ~seen_mask(n, n_k, window_left, window_right, prefix_len, sink_len)
        q = p.q[row:row + n].double().transpose(0, 1)
        s = (scale * q @ k.transpose(1, 2)).masked_fill(hidden, -np.inf)
        ref_l = torch.logsumexp(s, -1)
        w = torch.exp(s - ref_l[..., None])
        ref_o, a = w @ v, w @ v.abs()
        got_o, got_l = o[row:row + n].double().transpose(0, 1), lse[:, row:row + n].double()
        assert torch.isfinite(got_o).all() and torch.isfinite(got_l).all()
        size = (q.abs() @ k.abs().transpose(1, 2)).masked_fill(hidden, 0.0).amax(-1)
        lost = 2.0 ** -25 * q.abs().amax(-1) * (k.abs().sum(-1)[:, None].masked_fill(hidden, 0.0)).amax(-1)
        ds = abs(scale) * (1.07 * p.d * 2.0 ** -23 * size + lost)
        n_vis = (~hidden).sum(-1).double()[None, :]
        small = 2.0 ** -18 + 2.0 ** -23 * ve.abs().max()
        top = v.abs().amax(-1)
        unit = torch.where(top > 0, torch.clamp(top / 224, min=least), torch.zeros_like(top))
        floor = 2.0 ** -22 * (w * unit[:, None]).amax(-1)[..., None] * ((~hidden).double() @ vc.abs())
        tol = u * ref_o.abs() + denormal + floor + a * (2.0 ** -12 + 2 * ds + 2 * n_vis * 2.0 ** -23 + small)[..., None]
        worst = ((got_o - ref_o).abs() / tol.clamp(min=1e-300)).max()
        assert worst <= 1, "sequence %d: O off by %.2f tolerances" % (b, worst)
        worst = ((got_l - ref_l).abs() / (ds + n_vis * 2.0 ** -23 + small + 2.0 ** -22 * ref_l.abs())).max()
        assert worst <= 1, "sequence %d: L off by %.2f tolerances" % (b, worst)
        row += n


def fill(p, size, share, zeros, dtype, seed):
    """New rows for all of p's sequences: values of `size`, and zero rows at the keys that `zeros` names.  Of these the
    first has `share` of every row's weight; the others are ordinary keys."""
    g, dt, d = gen(seed), DT[dtype], p.d
    p.q.copy_(torch.randn(p.q.shape, generator=g, device="cuda") * 0.5)
    p.q[..., 0] = 4.0
    for b, n in enumerate(p.lens_k):
        k = torch.randn((n, p.hkv, d), generator=g, device="cuda")
        k[..., 0] = 0.0
        v = torch.randn((n, p.hkv, d), generator=g, device="cuda") * size
        at = [z % n for z in zeros]
        k[at[0]] = 0.0
        # the others' scores are normal, 0.5 in size: their sum is n e^(1/8)
        k[at[0], :, 0] = (np.log(share / (1 - share) * n) + 0.125) * d ** 0.5 / 4
        v[at] = 0.0
        fa2.fa2_paged_append_fp8(k.to(dt), v.to(dt), slots_of(p, b), *p.cache)


# (rows of a tile: up to 8, 16, 32, several tiles a sequence; pairs whole and cut)
SHAPES = {"8": ([1, 2], [2000, 300], 4), "8 cut": ([1], [30000], 4), "16": ([1, 2], [300, 2500], 8),
          "32": ([1, 1], [20000, 77], 32), "32 rows of 8 tokens": ([8, 3], [2000, 130], 4),
          "chunk": ([200, 1], [1500, 2500], 2), "many": ([1] * 40, [100 + 30 * b for b in range(40)], 4)}


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "bf16"), (256, "fp16"), (128, "fp16")])
@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("size,share", [(1.0, 0.9), (1e-2, 0.5), (1e-2, 0.99), (1e-3, 0.1)])
def test_a_zero_value_of_large_weight(share, size, shape, d, dtype):
    lens_q, lens_k, group = SHAPES[shape]
    p = Problem(lens_q, lens_k, group, 1, d, dtype, 16, seed=1)
    fill(p, size, share, [0], dtype, seed=2)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    check(p, o, lse)


@pytest.mark.parametrize("first", [5, 127, 128, 1000, -300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_zero_values_among_the_others(first, dtype):
    """The key of large weight in a later step than the first, and every seventh value zero beside it."""
    p = Problem([1, 3], [2000, 700], 8, 2, 128, dtype, 32, seed=3)
    fill(p, 0.02, 0.95, [first] + list(range(0, 700, 7)), dtype, seed=4)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    check(p, o, lse)


@pytest.mark.parametrize("mask", [dict(window_left=90, window_right=0, sink_len=4),
                                  dict(window_left=300, window_right=2, prefix_len=5),
                                  dict(window_left=700, window_right=0, sink_len=130)])
@pytest.mark.parametrize("lens_q,lens_k,group", [([1, 3], [2000, 600], 4), ([40, 1], [900, 1500], 3), ([2], [9000], 16)])
def test_zero_sinks_beside_a_window(lens_q, lens_k, group, mask):
    """The first keys, seen past the window's edge, hold most of the weight and zeros."""
    p = Problem(lens_q, lens_k, 2 * group, 2, 128, "bf16", 16, seed=11)
    fill(p, 0.02, 0.9, [0, 1, 2, 3], "bf16", seed=12)
    o, lse = p.run(**mask)
    assert status() == fa2.FA2_OK
    check(p, o, lse, **mask)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_all_values_zero(dtype):
    p = Problem([1, 3, 40], [2000, 700, 9000], 8, 2, 128, dtype, 32, seed=5)
    for b, n in enumerate(p.lens_k):
        k = torch.randn((n, 2, 128), generator=gen(b), device="cuda").to(DT[dtype])
        fa2.fa2_paged_append_fp8(k, torch.zeros_like(k).neg() if b else torch.zeros_like(k), slots_of(p, b), *p.cache)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    assert (o == 0).all()
    check(p, o, lse)


def test_zero_values_of_scores_that_rise():
    """Zero rows whose scores pass all before them on every step, up to 60 powers of two past the others'."""
    n, d = 3000, 64
    p = Problem([1], [n], 2, 1, d, "bf16", 16, seed=6)
    p.q.zero_()
    p.q[..., 0] = 1.0
    k = torch.zeros((n, 1, d), device="cuda")
    v = torch.randn((n, 1, d), generator=gen(7), device="cuda") * 0.01
    at = torch.arange(64, n, 128, device="cuda")
    k[at, 0, 0] = torch.linspace(1.0, 60.0, len(at), device="cuda") * np.log(2.0)
    v[at] = 0.0
    fa2.fa2_paged_append_fp8(k.bfloat16(), v.bfloat16(), slots_of(p, 0), *p.cache)
    o, lse = p.run(window_right=0, scale=1.0)
    assert status() == fa2.FA2_OK
    check(p, o, lse, scale=1.0)


def test_a_page_out_of_range_of_large_weight():
    """Its keys are zero codes: score 0, where the others' is -10."""
    p = Problem([1, 2], [600, 300], 4, 2, 128, "bf16", 16, seed=8)
    p.q.copy_(torch.randn(p.q.shape, generator=gen(9), device="cuda") * 0.5)
    p.q[..., 0] = 4.0
    for b, n in enumerate(p.lens_k):
        k = torch.randn((n, 2, 128), generator=gen(10 + b), device="cuda")
        k[..., 0] = -10 * 128 ** 0.5 / 4
        v = torch.randn((n, 2, 128), generator=gen(20 + b), device="cuda") * 0.02
        fa2.fa2_paged_append_fp8(k.bfloat16(), v.bfloat16(), slots_of(p, b), *p.cache)
    kept = p.table[0, 3].item()
    for bad in (-1, p.cache[0].shape[0]):
        p.table[0, 3] = bad
        o, lse = p.run(window_right=0)
        assert status() == fa2.FA2_ERR_DEVICE_PAGES
        p.table[0, 3] = kept
        saved = [x[kept].clone() for x in p.cache]
        p.cache[0].view(torch.uint8)[kept], p.cache[1].view(torch.uint8)[kept] = 0, 0
        p.cache[2][kept], p.cache[3][kept] = 127, 127
        check(p, o, lse)
        for x, y in zip(p.cache, saved):
            x.view(torch.uint8)[kept] = y.view(torch.uint8)
    assert status() == fa2.FA2_OK
