"""The paged key/value cache on the GPU: planning, appending and attention over
pages against plain implementations in 64 bits, alone and as serving steps.

Tolerances of the attention, per element, from the arithmetic (u = eps / 2 of
the 16-bit type, n the row's visible keys, A = sum p |v| its softmax-weighted
mean of |v|):
- O: P is rounded to 16 bits for the value product (u A) and O once (u |O|);
  a score sums d products in fp32, off by at most d 2^-23 scale sum |q k| (the
  tensor core may truncate its sums), which moves every p and their sum by that
  relative amount (2 dS A); P V and the row sum add n terms in fp32 (2 n 2^-23
  A); the exponential, the exp2-domain scale and the final division, and for
  split tiles the merge, stay below 2^-18 A.
- L: dS + n 2^-23 + 2^-18 + 2^-22 |L|.
Rows that see nothing are exactly O = 0, L = -inf; integers and copied rows are
equal bit for bit."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    fa2.load_library()
    yield
    code, detail = fa2.fa2_get_device_status()
    assert code == fa2.FA2_OK, "device status word set: 0x%x" % detail


def status():
    torch.cuda.synchronize()
    return fa2.fa2_get_device_status()[0]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def seen_mask(n_q, n_k, wl, wr, pre):
    i = torch.arange(n_q, device="cuda")[:, None] + (n_k - n_q)
    j = torch.arange(n_k, device="cuda")[None, :]
    seen = torch.ones((n_q, n_k), dtype=torch.bool, device="cuda")
    if wl >= 0:
        seen &= j >= i - wl
    if wr >= 0:
        seen &= j <= i + wr
    return seen | (j < pre)


class Problem:
    """Random queries and a cache of the given lengths, pages in random order."""

    def __init__(self, lens_q, lens_k, hq, hkv, d, dtype, page, seed, pages=None, table_extra=1, fill=None):
        self.lens_q, self.lens_k, self.page, self.d = list(lens_q), list(lens_k), page, d
        self.hq, self.hkv = hq, hkv
        g, dt = gen(seed), DT[dtype]
        need = [-(-n // page) for n in lens_k]
        pages = sum(need) + 2 if pages is None else pages
        order = torch.randperm(pages, generator=g, device="cuda")[:sum(need)].tolist()
        widest = max(need) + table_extra
        table = np.full((len(lens_k), max(widest, 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32).to(dt)
        total = max(1, sum(lens_q))
        self.q = rnd(total, hq, d)
        self.k = rnd(pages, hkv, page, d)
        self.v = rnd(pages, hkv, page, d)
        if fill is not None:   # rows no sequence holds: anything
            used = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
            for b, n in enumerate(lens_k):
                j = torch.arange(n, device="cuda")
                used[self.table[b, (j // page)].long(), j % page] = True
            for c in (self.k, self.v):
                c.copy_(torch.where(used[:, None, :, None], c, torch.full_like(c, fill)))
        self.cu = i32(np.concatenate([[0], np.cumsum(lens_q)]))
        self.lens = i32(lens_k)

    def run(self, **kw):
        kw.setdefault("max_seqlen_q", max(1, max(self.lens_q)))
        return fa2.fa2_paged_fwd(self.q, self.k, self.v, self.table, self.cu, self.lens, **kw)

    def check(self, o, lse, scale=None, window_left=-1, window_right=-1, prefix_len=0, skip=()):
        """Every output of every sequence against the definition in float64."""
        d, group = self.d, self.hq // self.hkv
        scale = 1.0 / d ** 0.5 if scale is None else scale
        u = torch.finfo(o.dtype).eps / 2
        row = 0
        for b, (n, n_k) in enumerate(zip(self.lens_q, self.lens_k)):
            if b in skip or n == 0:
                row += n
                continue
            j = torch.arange(n_k, device="cuda")
            pg = self.table[b, j // self.page].long()
            k = self.k[pg, :, j % self.page].double().transpose(0, 1)    # [hkv, n_k, d]
            v = self.v[pg, :, j % self.page].double().transpose(0, 1)
            k, v = (x.repeat_interleave(group, 0) for x in (k, v))
            q = self.q[row:row + n].double().transpose(0, 1)
            hidden = ~seen_mask(n, n_k, window_left, window_right, prefix_len)
            k, v = k.clone(), v.clone()
            dead = hidden.all(0)
            k[:, dead] = 0
            v[:, dead] = 0
            s = (scale * q @ k.transpose(1, 2)).masked_fill(hidden, -np.inf)
            ref_l = torch.logsumexp(s, -1) if n_k else torch.full(s.shape[:2], -np.inf, device="cuda").double()
            p = torch.exp(s - torch.where(torch.isinf(ref_l), torch.zeros_like(ref_l), ref_l)[..., None])
            ref_o = p @ v
            a = p @ v.abs()
            ds = (d * 2.0 ** -23) * abs(scale) * (q.abs() @ k.abs().transpose(1, 2)).amax(-1) if n_k else 0 * ref_l
            n_vis = (~hidden).sum(-1).double()[None, :]
            got_o = o[row:row + n].double().transpose(0, 1)
            got_l = lse[:, row:row + n].double()
            empty = torch.isinf(ref_l)
            assert torch.equal(torch.isneginf(got_l), empty), "sequence %d: rows without keys" % b
            assert (got_o[empty] == 0).all(), "sequence %d: a row without keys is not zero" % b
            tol_o = u * (a + ref_o.abs()) + a * (2 * ds + 2 * n_vis * 2.0 ** -23 + 2.0 ** -18)[..., None] + 1e-7
            worst = ((got_o - ref_o).abs() / tol_o)[~empty]
            assert torch.isfinite(got_o).all(), "sequence %d: non-finite output" % b
            assert worst.numel() == 0 or worst.max() <= 1, "sequence %d: O off by %.2f tolerances" % (b, worst.max())
            tol_l = ds + n_vis * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22 * ref_l.abs()
            worst = ((got_l - ref_l).abs() / tol_l)[~empty]
            assert worst.numel() == 0 or worst.max() <= 1, "sequence %d: L off by %.2f tolerances" % (b, worst.max())
            row += n


# (new tokens, keys) of the sequences: one token to chunks, empty ones, lengths around tiles and pages
BATCHES = {
    "decode": ([1] * 7, [1, 17, 64, 65, 700, 129, 4097]),
    "ragged": ([1, 0, 5, 130, 33, 1, 3, 64], [300, 40, 5, 131, 1000, 0, 2, 64]),
    "chunk": ([200, 1], [1500, 2500]),
}
MASKS = {"causal": (-1, 0, 0), "full": (-1, -1, 0), "window": (100, 0, 0), "sinks": (70, 0, 4), "wide": (130, 3, 100),
         "self": (0, 0, 0)}


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "fp16"), (64, "bf16"), (128, "fp16"),
                                     (256, "bf16")])
@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("batch", sorted(BATCHES))
def test_attention_against_definition(batch, mask, d, dtype):
    lens_q, lens_k = BATCHES[batch]
    page = {"decode": 16, "ragged": 8, "chunk": 64}[batch]
    group = {"decode": 4, "ragged": 3, "chunk": 1}[batch]
    p = Problem(lens_q, lens_k, 2 * group, 2, d, dtype, page, seed=d + len(batch), fill=float("nan"))
    wl, wr, pre = MASKS[mask]
    kw = dict(window_left=wl, window_right=wr, prefix_len=pre)
    o, lse = p.run(**kw)
    assert status() == fa2.FA2_OK
    p.check(o, lse, **kw)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 192, 1024])
@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 1), (5, 2), (7, 1), (8, 2), (16, 1), (33, 1), (128, 1)])
def test_page_sizes_and_groups(page, group, hkv):
    p = Problem([1, 9, 40, 1], [1025, 300, 40, 63], group * hkv, hkv, 128, "bf16", page, seed=page + group,
                fill=float("inf"))
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_any_finite_scale(d, scale):
    p = Problem([1, 6], [500, 90], 4, 2, d, "fp16", 16, seed=5, fill=float("nan"))
    o, lse = p.run(scale=scale, window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, scale=scale, window_right=0)


def test_many_sequences():
    """More sequences than threads of a block, a few long ones among them."""
    r = np.random.default_rng(3)
    lens_q = r.integers(0, 3, 1000).tolist()
    lens_k = [q + int(x) for q, x in zip(lens_q, r.integers(0, 90, 1000))]
    lens_k[500], lens_k[999], lens_q[999] = 9000, 7000, 40
    p = Problem(lens_q, lens_k, 4, 1, 64, "bf16", 16, seed=9)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)
    o2, lse2 = p.run(window_right=0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_many_decoding_sequences():
    """One to three tokens a sequence, more sequences than threads, some idle, some empty, a few long."""
    r = np.random.default_rng(4)
    lens_q = r.integers(0, 4, 1500).tolist()
    lens_k = [int(x) for x in r.integers(0, 200, 1500)]
    lens_k[3], lens_k[700], lens_k[1499], lens_q[1499] = 5000, 3000, 9000, 3
    p = Problem(lens_q, lens_k, 10, 2, 128, "bf16", 8, seed=14, fill=float("nan"))
    for kw in (dict(window_right=0), dict(window_left=90, window_right=0, prefix_len=3)):
        o, lse = p.run(**kw)
        assert status() == fa2.FA2_OK
        p.check(o, lse, **kw)


@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (128, "fp16"), (256, "bf16")])
@pytest.mark.parametrize("mask", sorted(MASKS))
def test_few_tokens_against_definition(mask, d, dtype):
    """Drafted tokens: several rows of each head, some before the sequence's first key."""
    p = Problem([7, 1, 8, 5, 3, 8], [1500, 3, 5, 64, 0, 4111], 10, 2, d, dtype, 32, seed=d + 1, fill=float("nan"))
    wl, wr, pre = MASKS[mask]
    kw = dict(window_left=wl, window_right=wr, prefix_len=pre)
    o, lse = p.run(**kw)
    assert status() == fa2.FA2_OK
    p.check(o, lse, **kw)


@pytest.mark.parametrize("batch,n_k,new", [(1, 300, 1), (3, 700, 2), (1, 100, 100), (30, 960, 1), (2, 5000, 64)])
def test_pairs_whole_and_cut(batch, n_k, new):
    """Around the rule that gives every (query tile, K/V head) pair a CTA of its own."""
    for hkv in (1, 8):
        p = Problem([new] * batch, [n_k] * batch, 4 * hkv, hkv, 128, "bf16", 64, seed=batch + n_k)
        o, lse = p.run(window_right=0)
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0)


def test_tables_wider_than_a_32_bit_line():
    """Table rows that could hold 2^31 keys each: few rows, but positions of the batch's work past 32 bits."""
    page, hkv, d, batch = 1 << 20, 2, 64, 64
    p = Problem([2] * batch, [130 + 7 * b for b in range(batch)], 4, hkv, d, "fp16", 64, seed=15)
    # the same keys in one page of 2^20 rows
    k = torch.zeros((1, hkv, page, d), dtype=torch.float16, device="cuda")
    v = torch.zeros_like(k)
    k[0, :, :700] = p.k[:11].transpose(0, 1).reshape(hkv, -1, d)[:, :700]
    v[0, :, :700] = p.v[:11].transpose(0, 1).reshape(hkv, -1, d)[:, :700]
    table = torch.full((batch, 2047), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    q = Problem.__new__(Problem)
    q.lens_q, q.lens_k, q.page, q.d, q.hq, q.hkv = p.lens_q, p.lens_k, page, d, 4, hkv
    q.q, q.k, q.v, q.table, q.cu, q.lens = p.q, k, v, table, p.cu, p.lens
    o, lse = q.run(window_right=0)
    assert status() == fa2.FA2_OK
    q.check(o, lse, window_right=0)


def test_many_query_tiles():
    """Prompts from their start: enough (query tile, K/V head) pairs for one CTA each, beside short sequences."""
    lens_q = [2500, 1, 1300, 7, 0, 900]
    lens_k = [2500, 900, 1300, 7, 5, 1000]
    p = Problem(lens_q, lens_k, 32, 8, 64, "fp16", 64, seed=13, fill=float("nan"))
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)
    o, lse = p.run(window_left=300, window_right=0, prefix_len=10)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_left=300, window_right=0, prefix_len=10)


@pytest.mark.parametrize("lens_q,lens_k", [
    ([1, 700, 0, 100], [900, 12800, 30, 13000]),   # the first wave ends inside a sequence,
    ([600, 100, 3], [13000, 13100, 500]),          # between two,
    ([90, 700, 128], [700, 13000, 128]),           # and over short ones
])
def test_full_waves_of_long_pairs(lens_q, lens_k):
    """Chunks whose keys outgrow the L2 cache: full waves of (query tile, K/V head) pairs run whole, the rest is cut."""
    p = Problem(lens_q, lens_k, 32, 8, 256, "fp16", 64, seed=14, fill=float("nan"))
    for kw in (dict(window_right=0), dict(window_right=3, prefix_len=100)):
        o, lse = p.run(**kw)
        assert status() == fa2.FA2_OK
        p.check(o, lse, **kw)


def test_layouts_equal_contiguous():
    """[page, row, head] caches, K and V interleaved, q and o as parts of wider rows, a sliced table."""
    p = Problem([3, 1, 70], [400, 33, 200], 8, 2, 128, "bf16", 16, seed=21)
    o, lse = p.run(window_right=0)
    kv = torch.empty((p.k.shape[0], 16, 2, 2, 128), dtype=p.k.dtype, device="cuda")   # page, row, k/v, head
    k, v = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    k.copy_(p.k)
    v.copy_(p.v)
    wide = torch.zeros((74, 8 + 4, 128), dtype=p.q.dtype, device="cuda")
    wide[:, 2:10] = p.q
    out = torch.full((74, 20, 128), 7.0, dtype=p.q.dtype, device="cuda")
    table = torch.full((3, 60), -9, dtype=torch.int32, device="cuda")
    table[:, 5:5 + p.table.shape[1]] = p.table
    lse_wide = torch.full((8, 100), 7.0, device="cuda")
    fa2.fa2_paged_fwd(wide[:, 2:10], k, v, table[:, 5:5 + p.table.shape[1]], p.cu, p.lens, o=out[:, 4:12],
                      lse=lse_wide[:, 20:94], window_right=0)
    assert status() == fa2.FA2_OK
    assert torch.equal(out[:, 4:12], o) and torch.equal(lse_wide[:, 20:94], lse)
    assert (out[:, :4] == 7).all() and (out[:, 12:] == 7).all()
    assert (lse_wide[:, :20] == 7).all() and (lse_wide[:, 94:] == 7).all()


@pytest.mark.parametrize("mask", ["causal", "sinks"])
@pytest.mark.parametrize("batch", [2, 31, 32, 33, 64])
def test_batches_around_one_sequence_a_lane(batch, mask):
    """Idle, empty, short and long sequences among up to 32 (a lane each) and more; then one of them out of range."""
    r = np.random.default_rng(batch)
    lens_q = r.integers(0, 4, batch).tolist()
    lens_k = [int(n) * int(r.integers(0, 9)) // 8 for n in r.integers(0, 3000, batch)]
    lens_q[-1], lens_k[-1] = 1, 1500
    wl, wr, pre = MASKS[mask]
    kw = dict(window_left=wl, window_right=wr, prefix_len=pre)
    p = Problem(lens_q, lens_k, 8, 2, 128, "bf16", 16, seed=batch, fill=float("nan"))
    o, lse = p.run(**kw)
    assert status() == fa2.FA2_OK
    p.check(o, lse, **kw)
    p.lens[batch - 1] = -1
    kept = torch.full_like(o, 3.0)
    o2, lse2 = p.run(o=kept, **kw)
    assert status() == fa2.FA2_ERR_DEVICE_SEQLENS
    p.check(o2, lse2, skip=[batch - 1], **kw)
    assert (o2[-1] == 3).all()


@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("lens_q,lens_k", [([5, 2, 9], [2, 0, 8]), ([200, 130, 1, 64], [50, 0, 0, 63]), ([300], [299])])
def test_more_tokens_than_keys(lens_q, lens_k, mask):
    """The first tokens come before every key: rows that see nothing, or only the prefix."""
    wl, wr, pre = MASKS[mask]
    p = Problem(lens_q, lens_k, 6, 2, 128, "bf16", 16, seed=23, fill=float("nan"))
    kw = dict(window_left=wl, window_right=wr, prefix_len=pre)
    o, lse = p.run(**kw)
    assert status() == fa2.FA2_OK
    p.check(o, lse, **kw)


def test_strides_of_single_dimensions_do_not_count():
    """One token, one head, one page, one sequence: whatever stride the dimension has."""
    p = Problem([1], [11], 1, 1, 64, "fp16", 16, seed=24, pages=1)
    o, lse = p.run(window_right=0)
    p.check(o, lse, window_right=0)
    odd = lambda x, st: torch.as_strided(x, x.shape, st, x.storage_offset())
    args = (odd(p.q, (3, 5, 1)), odd(p.k, (1, 7, 64, 1)), odd(p.v, (0, 1, 64, 1)), odd(p.table, (0, 1)), p.cu, p.lens)
    o2, lse2 = fa2.fa2_paged_fwd(*args, window_right=0)
    assert status() == fa2.FA2_OK
    assert torch.equal(o2, o) and torch.equal(lse2, lse)
    k, v = torch.zeros_like(p.k), torch.zeros_like(p.v)
    new = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda")
    fa2.fa2_paged_append(odd(new, (3, 5, 1)), new, i32([4]), odd(k, (1, 7, 64, 1)), v)
    assert status() == fa2.FA2_OK
    assert (k[0, 0, 4] == 1).all() and k.sum() == 64 and torch.equal(k, v)


@pytest.mark.parametrize("new", [1, 40])
def test_sequences_sharing_one_table_row(new):
    """A prompt's pages read by several sequences through one row (stride 0), each with its own length."""
    p = Problem([new] * 5, [700, 64, 333, 80, 699], 8, 2, 128, "bf16", 16, seed=25)
    shared = p.table[:1].expand(5, -1)
    q = Problem.__new__(Problem)
    q.__dict__.update(p.__dict__)
    q.table = shared
    o, lse = q.run(window_right=0)
    assert status() == fa2.FA2_OK
    q.check(o, lse, window_right=0)


def test_two_forwards_at_once():
    """Long and short calls overlapping on two streams, few and many rows, each with its own workspace."""
    probs = [Problem([1] * 40, [2000 + 37 * i for i in range(40)], 16, 4, 128, "bf16", 16, seed=26),
             Problem([300, 77], [5000, 900], 16, 4, 128, "bf16", 64, seed=27)]
    want = [p.run(window_right=0) for p in probs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in probs]
    outs = [[], []]
    for _ in range(20):
        for p, st, out in zip(probs, streams, outs):
            out.append(p.run(window_right=0, stream=st))
    assert status() == fa2.FA2_OK
    for p, (wo, wl), out in zip(probs, want, outs):
        p.check(wo, wl, window_right=0)
        for o, lse in out:
            assert torch.equal(o, wo) and torch.equal(lse, wl)


def test_padded_pages():
    """Page strides that are no whole number of head strides (pages padded apart), in K, in V and in both."""
    p = Problem([3, 1, 70], [400, 33, 200], 6, 3, 64, "fp16", 32, seed=22)
    o, lse = p.run(window_right=0)
    for which in ("k", "v", "kv"):
        side = {}
        for name, src in (("k", p.k), ("v", p.v)):
            n = src[0].numel()
            wide = torch.full((src.shape[0], n + 8), float("nan"), dtype=src.dtype, device="cuda")
            wide[:, :n] = src.reshape(src.shape[0], n)
            side[name] = wide[:, :n].unflatten(1, src.shape[1:]) if name in which else src
        o2, lse2 = fa2.fa2_paged_fwd(p.q, side["k"], side["v"], p.table, p.cu, p.lens, window_right=0, max_seqlen_q=70)
        assert status() == fa2.FA2_OK
        assert torch.equal(o2, o) and torch.equal(lse2, lse)


def test_pages_no_query_sees_are_not_read():
    """Pages before a sliding window may be gone: entries out of range, their rows NaN."""
    page, n_k = 16, 1000
    p = Problem([1, 30], [n_k, n_k], 4, 1, 64, "fp16", page, seed=31)
    for pre in (0, 4):
        q = Problem([1, 30], [n_k, n_k], 4, 1, 64, "fp16", page, seed=31)
        for b, n in enumerate((1, 30)):
            first = (n_k - n - 100) // page   # first page the window reaches
            for e in range(1 if pre else 0, first):
                q.k[q.table[b, e].long()] = float("nan")
                q.v[q.table[b, e].long()] = float("nan")
                q.table[b, e] = (-1, 10 ** 9)[e % 2]
        kw = dict(window_left=100, window_right=0, prefix_len=pre)
        o, lse = q.run(**kw)
        assert status() == fa2.FA2_OK
        want, want_l = p.run(**kw)
        assert torch.equal(o, want) and torch.equal(lse, want_l)
        p.check(o, lse, **kw)


def test_rows_outside_sequences_are_left():
    p = Problem([2, 1, 5], [20, 3, 70], 4, 2, 128, "fp16", 32, seed=41)
    q = torch.cat([p.q, torch.full((6, 4, 128), float("nan"), dtype=p.q.dtype, device="cuda")])
    o = torch.full_like(q, 3.0)
    lse = torch.full((4, 14), 3.0, device="cuda")
    fa2.fa2_paged_fwd(q, p.k, p.v, p.table, p.cu, p.lens, o=o, lse=lse, window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o[:8], lse[:, :8], window_right=0)
    assert (o[8:] == 3).all() and (lse[:, 8:] == 3).all()


def test_bad_sequences_are_left_and_reported():
    p = Problem([2, 1, 5, 1], [20, 3, 70, 9], 4, 2, 64, "bf16", 16, seed=51)
    cap = p.table.shape[1] * 16
    for lens, cu, bad in (([20, -1, 70, cap + 1], [0, 2, 3, 8, 9], (1, 3)),
                          ([20, 3, 70, 9], [0, 2, 3, 8, 10], (3,)),        # past total_q
                          ([20, 3, 70, 9], [-1, 2, 3, 8, 9], (0,))):
        o = torch.full_like(p.q, 3.0)
        lse = torch.full((4, 9), 3.0, device="cuda")
        fa2.fa2_paged_fwd(p.q, p.k, p.v, p.table, i32(cu), i32(lens), o=o, lse=lse, window_right=0)
        assert status() == fa2.FA2_ERR_DEVICE_SEQLENS
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0, skip=bad)
        for b in bad:
            assert (o[(0, 2, 3, 8)[b]:(2, 3, 8, 9)[b]] == 3).all()
            assert (lse[:, (0, 2, 3, 8)[b]:(2, 3, 8, 9)[b]] == 3).all()
    fa2.fa2_paged_fwd(p.q, p.k, p.v, p.table, p.cu, p.lens, window_right=0, max_seqlen_q=4)   # one has 5
    assert status() == fa2.FA2_ERR_DEVICE_SEQLENS


def test_needed_page_out_of_range_reads_as_zeros():
    p = Problem([1, 40], [100, 100], 2, 1, 128, "bf16", 16, seed=61)
    want = Problem([1, 40], [100, 100], 2, 1, 128, "bf16", 16, seed=61)
    for b, e, page in ((0, 2, -1), (1, 0, p.k.shape[0]), (1, 3, 2 ** 31 - 1), (1, 4, -2 ** 31)):
        want.k[p.table[b, e].long()] = 0
        want.v[p.table[b, e].long()] = 0
        p.table[b, e] = page
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    want.check(o, lse, window_right=0)


def test_cache_beyond_32_bit_offsets():
    """K and V in one allocation of 2^32 elements; the pages used lie at its end."""
    page, hkv, d = 64, 4, 128
    pages = 2 ** 31 // (page * hkv * d) + 40
    kv = torch.empty((pages, 2, hkv, page, d), dtype=torch.bfloat16, device="cuda")
    p = Problem([1, 33], [1000, 500], 8, hkv, d, "bf16", page, seed=71)
    kv[-40:].zero_()
    base = pages - p.k.shape[0]
    kv[base:, 0], kv[base:, 1] = p.k, p.v
    table = torch.where(p.table >= 0, p.table + base, p.table)
    o, lse = fa2.fa2_paged_fwd(p.q, kv[:, 0], kv[:, 1], table, p.cu, p.lens, window_right=0, max_seqlen_q=33)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)
    rows = torch.randn((34, hkv, d), device="cuda").bfloat16()
    slots = i32([(pages - 1) * page + 63 - i for i in range(34)])
    fa2.fa2_paged_append(rows, rows + 1, slots, kv[:, 0], kv[:, 1])
    assert status() == fa2.FA2_OK
    at = torch.arange(63, 29, -1, device="cuda")
    assert torch.equal(kv[-1, 0][:, at].transpose(0, 1), rows)
    assert torch.equal(kv[-1, 1][:, at].transpose(0, 1), rows + 1)


def test_agrees_with_the_contiguous_forward():
    """One page table over contiguous keys: the general forward's inputs, within both calls' rounding."""
    n_q, n_k, h, d = 100, 640, 4, 128
    p = Problem([n_q], [n_k], h, h, d, "bf16", 64, seed=81)
    k, v = (c[p.table[0, :10].long()].transpose(0, 1).reshape(1, h, n_k, d) for c in (p.k, p.v))
    o, lse = p.run(window_right=0)
    o2, lse2 = fa2.fa2_fwd_ex(p.q.transpose(0, 1)[None], k, v, window_left=-1, window_right=0)
    assert status() == fa2.FA2_OK
    assert (o.double() - o2[0].transpose(0, 1).double()).abs().max() <= 2 ** -8 * 2 * o2.double().abs().max()
    assert (lse - lse2[0]).abs().max() <= 1e-5


# ---------------------------------------------------------------- planning and appending


def plan_reference(ctx, new, table, free, count, page, total):
    table, stack = table.copy(), list(free[:count])
    cu, slots = [0], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        for pos in range(c, c + n):
            if pos % page == 0:
                table[b, pos // page] = stack.pop()
            slots.append(int(table[b, pos // page]) * page + pos % page)
        cu.append(cu[-1] + n)
    return cu, [c + n for c, n in zip(ctx, new)], slots + [-1] * (total - len(slots)), len(stack), table


@pytest.mark.parametrize("page", [1, 8, 16, 100, 256])
@pytest.mark.parametrize("batch,top,pad", [(1, 1, 0), (1, 5000, 3), (7, 40, 0), (300, 1, 9), (2500, 30, 1), (16384, 3, 0)])
def test_plan_against_reference(batch, top, pad, page):
    r = np.random.default_rng(batch + top + page)
    ctx = r.integers(0, 3 * page + 50, batch)
    new = r.integers(0, top + 1, batch)
    new[0] = top
    held = -(-ctx // page)
    need = -(-(ctx + new) // page)
    pages = int(need.sum()) + 5
    order = r.permutation(pages).astype(np.int32)
    width = int(need.max()) + 2
    table = np.full((batch, width), -7, np.int32)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.concatenate([order[at:], np.full(11, -1, np.int32)])   # beyond the count: not read
    count, total = pages - at, max(1, int(new.sum()) + pad)
    want = plan_reference(ctx.tolist(), new.tolist(), table, free.tolist(), count, page, total)
    wide = torch.full((batch, width + 3), -5, dtype=torch.int32, device="cuda")
    wide[:, :width] = torch.from_numpy(table).cuda()
    args = (i32(ctx), i32(new), wide[:, :width], torch.from_numpy(free).cuda(), i32([count]), pages, page, total)
    for _ in range(2):   # the count is read, not written: a second call gives the same step
        cu, lens, slots, left = fa2.fa2_paged_plan(*args)
        assert status() == fa2.FA2_OK
        assert cu.tolist() == want[0] and lens.tolist() == want[1] and slots.tolist() == want[2]
        assert left.item() == want[3]
        assert np.array_equal(wide[:, :width].cpu().numpy(), want[4])
        assert (wide[:, width:] == -5).all()


@pytest.mark.parametrize("why", ["pages", "negative", "negative new", "width", "rows", "count", "count below"])
def test_plan_refuses_a_step_whole(why):
    ctx, new, count, total = [5, 30, 0], [4, 1, 70], 9, 80
    if why == "pages":
        count = 5                       # needs 1 + 0 + 5
    if why == "negative":
        ctx[0] = -1
    if why == "negative new":
        new[1] = -2 ** 31
    if why == "width":
        new[2] = 16 * 6 + 1
    if why == "rows":
        total = 74
    if why == "count":
        count = 21
    if why == "count below":
        count = -1
    ctx[0] = 16 if why == "pages" else ctx[0]
    table = torch.arange(18, dtype=torch.int32, device="cuda").reshape(3, 6)
    keep = table.clone()
    free = torch.arange(20, 40, dtype=torch.int32, device="cuda")
    cu, lens, slots, left = fa2.fa2_paged_plan(i32(ctx), i32(new), table, free, i32([count]), 64, 16, total)
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    assert torch.equal(table, keep) and left.item() == count
    assert (cu == 0).all() and (lens == 0).all() and (slots == -1).all()
    # the step does nothing: no row appended, no output written
    cache = torch.zeros((64, 1, 16, 64), dtype=torch.float16, device="cuda")
    rows = torch.ones((total, 1, 64), dtype=torch.float16, device="cuda")
    v_cache = cache.clone()
    fa2.fa2_paged_append(rows, rows, slots, cache, v_cache)
    o = torch.full((total, 2, 64), 3.0, dtype=torch.float16, device="cuda")
    fa2.fa2_paged_fwd(rows.expand(total, 2, 64).contiguous(), cache, v_cache, table, cu, lens, o=o, window_right=0)
    assert status() == fa2.FA2_OK
    assert (cache == 0).all() and (v_cache == 0).all() and (o == 3).all()


@pytest.mark.parametrize("count,code", [(1, fa2.FA2_OK), (0, fa2.FA2_ERR_DEVICE_PAGES)])
def test_plan_of_almost_2_31_rows(count, code):
    """Padding whose row numbers end just below 2^31, in a step that fits and in one that is refused."""
    total = 2 ** 31 - 1000
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    cu, lens, slots, left = fa2.fa2_paged_plan(i32([0, 0]), i32([3, 0]), table, i32([7]), i32([count]), 9, 16, total)
    assert status() == code
    assert slots[:3].tolist() == ([112, 113, 114] if count else [-1] * 3)
    assert slots[3:].max().item() == -1 and slots[3:].min().item() == -1
    assert cu.tolist() == ([0, 3, 3] if count else [0, 0, 0]) and left.item() == 0


def test_plan_reports_bad_pages():
    # the held partial page of request 0 and the first page taken are out of range: their tokens get no slot
    table = i32([[64, -1, -1], [3, -1, -1]])
    cu, lens, slots, left = fa2.fa2_paged_plan(i32([15, 16]), i32([2, 1]), table, i32([9, 8, -4]), i32([3]), 64, 16, 4)
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    assert slots.tolist() == [-1, -1, 8 * 16, -1] and left.item() == 1 and cu.tolist() == [0, 2, 3]


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("hkv,page,total", [(1, 8, 1), (8, 16, 64), (3, 64, 100), (40, 192, 700)])
def test_append_against_indexing(hkv, page, total, d, dtype):
    g = gen(total + d)
    pages = total // page + 3
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:total].to(torch.int32)
    slots[total // 2::7] = -1
    rows = torch.randn((total, 3 * hkv, d), generator=g, device="cuda").to(DT[dtype])
    k, v = rows[:, hkv:2 * hkv], rows[:, 2 * hkv:]
    kc = torch.randn((pages, hkv, page, d), generator=g, device="cuda").to(DT[dtype])
    vc = torch.randn((pages, page, hkv, d), generator=g, device="cuda").to(DT[dtype]).transpose(1, 2)
    wk, wv = kc.clone(), vc.clone()
    keep = slots >= 0
    s = slots[keep].long()
    wk[s // page, :, s % page] = k[keep]
    wv[s // page, :, s % page] = v[keep]
    fa2.fa2_paged_append(k, v, slots, kc, vc)
    assert status() == fa2.FA2_OK
    assert torch.equal(kc, wk) and torch.equal(vc, wv)
    fa2.fa2_paged_append(k, v, torch.full_like(slots, pages * page), kc, vc)   # past the cache: skipped, reported
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


@pytest.mark.parametrize("total", [8191, 8192, 20000])
def test_append_of_many_rows(total):
    """Around 32 MB of rows, from which on they pass the L2 by."""
    g = gen(total)
    hkv, d, page = 8, 128, 64
    pages = total // page + 2
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:total].to(torch.int32)
    slots[::5] = -1
    rows = torch.randint(-2 ** 15, 2 ** 15, (total, 2, hkv, d), generator=g, device="cuda", dtype=torch.int16)
    rows = rows.view(torch.bfloat16)   # any bits
    kc, vc = (torch.zeros((pages, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa2.fa2_paged_append(rows[:, 0], rows[:, 1], slots, kc, vc)
    assert status() == fa2.FA2_OK
    keep = slots >= 0
    s = slots[keep].long()
    for i, cache in enumerate((kc, vc)):
        want = torch.zeros_like(cache)
        want[s // page, :, s % page] = rows[keep, i]
        assert torch.equal(cache.view(torch.int16), want.view(torch.int16))


# ---------------------------------------------------------------- serving steps


class Server:
    """A cache, its free list and the requests' tokens on the host, for checking."""

    def __init__(self, batch, hq, hkv, d, dtype, page, pages, width, total, seed):
        self.g, self.dt = gen(seed), DT[dtype]
        self.hq, self.hkv, self.d, self.page, self.pages = hq, hkv, d, page, pages
        nan = lambda: torch.full((pages, hkv, page, d), float("nan"), dtype=self.dt, device="cuda")
        self.k, self.v = nan(), nan()
        self.table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=self.g, device="cuda").to(torch.int32)
        self.count, self.ctx = i32([pages]), i32([0] * batch)
        self.total = total
        self.kept = [[] for _ in range(batch)]   # (k, v) rows of each request
        z = lambda h: torch.zeros((total, h, d), dtype=self.dt, device="cuda")
        self.q, self.nk, self.nv, self.new = z(hq), z(hkv), z(hkv), i32([0] * batch)

    def inputs(self, new):
        self.new.copy_(i32(new))
        for t in (self.q, self.nk, self.nv):
            t.copy_(torch.randn(t.shape, generator=self.g, device="cuda").to(self.dt))
        at = 0
        for b, n in enumerate(new):
            self.kept[b].append((self.nk[at:at + n].clone(), self.nv[at:at + n].clone()))
            at += n

    def step(self, max_q, **kw):
        """The calls of one serving step; the lengths stay on the GPU."""
        cu, lens, slots, left = fa2.fa2_paged_plan(self.ctx, self.new, self.table, self.free, self.count, self.pages,
                                                   self.page, self.total)
        fa2.fa2_paged_append(self.nk, self.nv, slots, self.k, self.v)
        out = fa2.fa2_paged_fwd(self.q, self.k, self.v, self.table, cu, lens, window_right=0, max_seqlen_q=max_q, **kw)
        self.ctx.copy_(lens)
        self.count.copy_(left)
        return out

    def check(self, o, lse, new):
        """Against attention over the requests' own rows, kept apart from the cache."""
        lens = [sum(x[0].shape[0] for x in rows) for rows in self.kept]
        p = Problem.__new__(Problem)
        p.lens_q, p.lens_k, p.page, p.d, p.hq, p.hkv, p.q = list(new), lens, max(lens), self.d, self.hq, self.hkv, self.q
        side = lambda i: torch.stack([torch.nn.functional.pad(torch.cat([x[i] for x in rows]),
                                                              (0, 0, 0, 0, 0, max(lens) - n)).transpose(0, 1)
                                      for rows, n in zip(self.kept, lens)])
        p.k, p.v = side(0), side(1)      # one page per request
        p.table = torch.arange(len(lens), dtype=torch.int32, device="cuda")[:, None]
        p.check(o, lse, window_right=0)


STEPS = [[70, 3, 0, 200], [1, 1, 33, 1], [1, 0, 1, 1], [1, 1, 1, 40], [15, 1, 1, 1]]


@pytest.mark.parametrize("d,dtype,page", [(128, "bf16", 16), (64, "fp16", 64), (256, "fp16", 8)])
def test_serving_steps(d, dtype, page):
    s = Server(4, 6, 2, d, dtype, page, pages=600 // page + 8, width=400 // page + 2, total=280, seed=page)
    for new in STEPS:
        s.inputs(new)
        o, lse = s.step(max_q=200)
        assert status() == fa2.FA2_OK
        s.check(o, lse, new)
    assert s.count.item() == s.pages - sum(-(-sum(x[0].shape[0] for x in rows) // page) for rows in s.kept)


def test_captured_step_replays_with_new_lengths():
    """One captured step replayed for every step of a run, and two graphs sharing a workspace."""
    s = Server(4, 6, 2, 128, "bf16", 16, pages=50, width=30, total=280, seed=1)
    need = fa2.fa2_paged_fwd_workspace_bytes(s.q, s.k, s.v, s.table, i32([0] * 5), i32([0] * 4), max_seqlen_q=200)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    s.step(max_q=200, workspace=ws)   # an idle step: nothing new
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s.step(max_q=200, workspace=ws)
        graphs.append((graph, out))
    for i, new in enumerate(STEPS):
        s.inputs(new)
        graph, (o, lse) = graphs[i % 2]
        graph.replay()
        assert status() == fa2.FA2_OK
        s.check(o, lse, new)


@pytest.mark.parametrize("captured", [False, True])
def test_step_forked_over_streams(captured):
    """A step whose rows are appended in halves on two streams between the plan and the forward."""
    s = Server(4, 6, 2, 128, "bf16", 16, pages=50, width=30, total=280, seed=2)
    sides = [torch.cuda.Stream() for _ in range(2)]

    def step():
        cu, lens, slots, left = fa2.fa2_paged_plan(s.ctx, s.new, s.table, s.free, s.count, s.pages, s.page, s.total)
        here = torch.cuda.current_stream()
        for i, side in enumerate(sides):
            part = slice(i * 140, i * 140 + 140)
            side.wait_stream(here)
            fa2.fa2_paged_append(s.nk[part], s.nv[part], slots[part], s.k, s.v, stream=side)
        for side in sides:
            here.wait_stream(side)
        out = fa2.fa2_paged_fwd(s.q, s.k, s.v, s.table, cu, lens, window_right=0, max_seqlen_q=200)
        s.ctx.copy_(lens)
        s.count.copy_(left)
        return out

    step()   # an idle step
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = step()
    for new in STEPS:
        s.inputs(new)
        if captured:
            graph.replay()
        else:
            torch.cuda.synchronize()
            o, lse = step()
        assert status() == fa2.FA2_OK
        s.check(o, lse, new)


def test_side_streams():
    """Calls on streams of their own, results and workspaces allocated there."""
    probs = [Problem([1] * 8, [3000 + 100 * i] * 8, 8, 2, 128, "bf16", 16, seed=i) for i in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in probs]
    outs = [[] for _ in probs]
    for _ in range(5):
        for p, st, out in zip(probs, streams, outs):
            out.append(p.run(window_right=0, stream=st))
    assert status() == fa2.FA2_OK
    for p, out in zip(probs, outs):
        want = p.run(window_right=0)
        p.check(*want, window_right=0)
        for o, lse in out:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_binding_refuses_mismatches():
    p = Problem([1], [20], 4, 2, 64, "fp16", 16, seed=1)
    good = dict(q=p.q, k_cache=p.k, v_cache=p.v, block_table=p.table, cu_seqlens_q=p.cu, seqlens_k=p.lens)
    for bad, err in ((dict(q=p.q.bfloat16()), TypeError), (dict(q=p.q.cpu()), ValueError), (dict(q=p.q[:, :3]), fa2.Fa2Error),
                     (dict(v_cache=p.v[:1]), ValueError), (dict(block_table=p.table.long()), ValueError),
                     (dict(seqlens_k=i32([1, 2])), ValueError), (dict(cu_seqlens_q=p.cu[:1]), ValueError),
                     (dict(o=torch.empty_like(p.q).float()), ValueError), (dict(lse=torch.empty((1, 4), device="cuda")), ValueError),
                     (dict(k_cache=p.k[..., :32], v_cache=p.v[..., :32], q=p.q[..., :32]), fa2.Fa2Error),
                     (dict(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda")), fa2.Fa2Error)):
        with pytest.raises(err):
            fa2.fa2_paged_fwd(**dict(good, **bad))
    with pytest.raises(ValueError):
        fa2.fa2_paged_append(p.k[:, :, 0], p.v[:, :, 0], i32([0]), p.k, p.v)
    with pytest.raises(ValueError):
        fa2.fa2_paged_plan(i32([1]), i32([1, 2]), p.table, i32([3]), i32([1]), 4, 16, 1)
