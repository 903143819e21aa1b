"""The paged key/value cache of 8-bit rows on the GPU: quantising rows as they
are written, reading them back, and attention that reads the pages in place,
against plain implementations in 64 bits.

Codes, exponents and rows read back are equal bit for bit (one rounding each,
of exactly known values).  Tolerances of the attention, per element, from the
arithmetic (u = eps / 2 of the 16-bit type, n the row's visible keys, v = code
2^e a value, A = sum p |v|):
- O is rounded once (u |O|).  P 2^e goes to the value product as three e4m3
  parts, each within 2^-4 of what the one before left: 2^-12 A; the third part's
  smallest step, 2^-9 at a scale of 2^-8, rounds by 2^-18 where the row's largest
  P 2^e is at least 2^4: 2^-22 max(p 2^e) sum |code|.  A score sums d products in
  fp32, off by at most d 2^-23 scale sum |q k| for the first part of q and 1/16
  and 1/256 of that for the others (1.07 in all); what q's third part rounds
  away is 2^-25 of the row's largest |q|.  The score moves P by that relative
  amount, and their sum (2 dS A).  P V and the row sum add n terms in fp32 (2 n
  2^-23 A); exponential, exponents added in the exp2 domain (2^-23 max |e|),
  division and merge: 2^-18 + 2^-23 max |e|.
- L: dS + n 2^-23 + 2^-18 + 2^-23 max |e| + 2^-22 |L|."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
LIMITS = {torch.float16: (-15, 8), torch.bfloat16: (-60, 60)}


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
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------- the format, in numpy

def code_values():
    """The 256 e4m3 values by code; 0x7f and 0xff are NaN."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    x = np.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7.0))
    x = np.where(c & 128, -x, x)
    x[(c & 127) == 127] = np.nan
    return x


VALUES = code_values()


def quantise(rows, dtype):
    """(codes, exponent bytes) of float64 rows [..., d] by search over all codes."""
    lo, hi = LIMITS[dtype]
    x = np.clip(rows, -240.0 * 2.0 ** hi, 240.0 * 2.0 ** hi)
    top = np.nan_to_num(np.abs(x), nan=0.0).max(-1)
    e = np.full(top.shape, lo)
    for k in range(lo, hi):
        e = np.where(top > 448.0 * 2.0 ** k, k + 1, e)
    e = np.where(top == 0, 0, e)
    y = np.abs(x) * 2.0 ** -e[..., None].astype(np.float64)
    grid = VALUES[:127]
    at = np.searchsorted(grid, np.nan_to_num(y, nan=0.0)).clip(1, 126)
    down, up = grid[at - 1], grid[at]
    near = np.where((y - down < up - y) | ((y - down == up - y) & ((at - 1) % 2 == 0)), at - 1, at)
    code = np.where(np.isnan(x), 127, near + np.where(np.signbit(x), 128, 0))
    return code.astype(np.uint8), (e + 127).astype(np.uint8)


def new_cache(pages, hkv, page, d, fill=0):
    codes = [torch.full((pages, hkv, page, d), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)]
    exps = [torch.full((pages, hkv, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    return codes + exps


def rows_of(g, shape, dt):
    """Rows whose sizes differ."""
    size = torch.exp(0.7 * torch.randn(shape[:-1], generator=g, device="cuda"))
    return (torch.randn(shape, generator=g, device="cuda") * size[..., None]).to(dt)


# ---------------------------------------------------------------- writing and reading back

@pytest.mark.parametrize("total", [1, 2, 77, 1030])
@pytest.mark.parametrize("hkv,d,page", [(1, 64, 8), (3, 128, 16), (8, 256, 64), (2, 64, 192), (5, 128, 32)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_quantised_and_read_back(total, hkv, d, page, dtype):
    dt = DT[dtype]
    g = gen(total + d)
    pages = (total + page - 1) // page + 2
    k, v = rows_of(g, (total, hkv, d), dt), rows_of(g, (total, hkv, d), dt)
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:total].to(torch.int32)
    slots[total // 2] = -1
    cache = new_cache(pages, hkv, page, d, fill=0x35)
    before = [x.clone() for x in cache]
    fa2.fa2_paged_append_fp8(k, v, slots, *cache)
    back = [torch.full((total, hkv, d), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    out = fa2.fa2_paged_read_fp8(slots, *cache, k=back[0], v=back[1])
    assert out[0] is back[0] and out[1] is back[1]
    other = fa2.fa2_paged_read_fp8(slots, *cache, dtype=torch.bfloat16)
    assert status() == fa2.FA2_OK
    keep = np.arange(total) != total // 2
    at = slots.cpu().numpy()[keep]
    for i, x in enumerate((k, v)):
        code, e = quantise(x.double().cpu().numpy()[keep], dt)
        want_c = before[i].view(torch.uint8).cpu().numpy().copy()
        want_e = before[2 + i].cpu().numpy().copy()
        want_c[at // page, :, at % page] = code
        want_e[at // page, :, at % page] = e
        assert np.array_equal(cache[i].view(torch.uint8).cpu().numpy(), want_c)
        assert np.array_equal(cache[2 + i].cpu().numpy(), want_e)
        value = VALUES[code] * 2.0 ** (e.astype(np.float64) - 127)[..., None]
        assert np.array_equal(back[i].double().cpu().numpy()[keep], value)   # exact in the rows' own type
        assert np.array_equal(other[i].double().cpu().numpy()[keep], value)  # and in bf16
        assert (back[i][total // 2] == 7).all()                              # a skipped row is left


@pytest.mark.parametrize("d,hkv", [(64, 16), (128, 9), (256, 4)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_rows_as_few_rows_at_a_time(d, hkv, dtype):
    """One call for a long prompt's rows (special values, skipped and bad slots among them) leaves what calls of 500 leave."""
    total, page = 4200, 16
    g = gen(d)
    k, v = rows_of(g, (total, hkv, d), DT[dtype]), rows_of(g, (total, hkv, d), DT[dtype])
    k[7, 0, 3], k[4000, 1], v[4100, 0, 0], v[11, 1, 5] = float("nan"), 0.0, float("inf"), -6e4
    pages = total // page + 1
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:total].to(torch.int32)
    slots[3000], slots[4150] = -1, pages * page
    one, many = (new_cache(pages, hkv, page, d, fill=0x35) for _ in range(2))
    fa2.fa2_paged_append_fp8(k, v, slots, *one)
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    for i in range(0, total, 500):
        fa2.fa2_paged_append_fp8(k[i:i + 500], v[i:i + 500], slots[i:i + 500], *many)
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    for x, y in zip(one, many):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_every_16_bit_value_is_rounded_to_its_nearest_code(dtype):
    """All 65536 values of the type, in rows whose exponent a 448-sized head value fixes, then by themselves."""
    dt = DT[dtype]
    every = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.uint16).view(dt)
    rows = every.reshape(1024, 1, 64).clone()
    lead = rows.clone()
    lead[..., 0] = 448.0
    for x in (rows, lead):
        cache = new_cache(64, 1, 16, 64)
        slots = torch.arange(1024, dtype=torch.int32, device="cuda")
        fa2.fa2_paged_append_fp8(x, x, slots, *cache)
        ref = x.double().cpu().numpy().reshape(64, 16, 64)[:, None]
        code, e = quantise(ref, dt)
        got = cache[0].view(torch.uint8).cpu().numpy()
        nan = np.isnan(ref)
        assert np.array_equal(got[~nan], code[~nan]) and ((got[nan] & 127) == 127).all()
        assert np.array_equal(cache[2].cpu().numpy(), e) and np.array_equal(cache[3].cpu().numpy(), e)
        k, _ = fa2.fa2_paged_read_fp8(slots, *cache, dtype=dt)
        value = VALUES[code] * 2.0 ** (e.astype(np.float64) - 127)[..., None]
        got = k.double().cpu().numpy().reshape(64, 16, 64)[:, None]
        assert np.array_equal(got[~nan], value[~nan]) and np.isnan(got[nan]).all()
    assert status() == fa2.FA2_OK


def test_rows_of_zeros_and_special_values():
    x = torch.zeros((6, 1, 128), dtype=torch.bfloat16, device="cuda")
    x[1, 0, 5] = 1.0
    x[2, 0, 5] = float("inf")
    x[3, 0, 5] = float("nan")
    x[3, 0, 6] = -3.0
    x[4] = 1e-30
    x[5, 0, 0], x[5, 0, 1] = -3e38, 1.0
    cache = new_cache(1, 1, 8, 128)
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    fa2.fa2_paged_append_fp8(x, x, slots, *cache)
    k, _ = fa2.fa2_paged_read_fp8(slots, *cache)
    assert status() == fa2.FA2_OK
    assert cache[2][0, 0, :6].tolist() == [127, 127 - 8, 187, 127 - 7, 67, 187]
    assert (k[0] == 0).all() and (k[4] == 0).all()
    assert k[1, 0, 5] == 1 and k[2, 0, 5] == 240 * 2.0 ** 60 and k[5, 0, 0] == -240 * 2.0 ** 60
    assert torch.isnan(k[3, 0, 5]) and k[3, 0, 6] == -3 and torch.isnan(k[3, 0]).sum() == 1


def test_fp16_rows_read_as_bf16_and_bf16_rows_as_fp16():
    g = gen(3)
    x = rows_of(g, (9, 2, 64), torch.bfloat16)
    x[0, 0, 0] = 3e5   # past fp16
    cache = new_cache(2, 2, 8, 64)
    slots = torch.arange(9, dtype=torch.int32, device="cuda")
    fa2.fa2_paged_append_fp8(x, x, slots, *cache)
    b, _ = fa2.fa2_paged_read_fp8(slots, *cache)
    h, _ = fa2.fa2_paged_read_fp8(slots, *cache, dtype=torch.float16)
    assert b.dtype == torch.bfloat16 and h.dtype == torch.float16
    assert torch.equal(h, b.float().half())
    assert torch.isinf(h[0, 0, 0])


@pytest.mark.parametrize("layout", ["pages_rows_heads", "interleaved", "one_allocation"])
def test_layouts_of_the_cache(layout):
    """Strided caches give the same codes, rows and attention as contiguous ones."""
    pages, hkv, page, d, total = 9, 2, 16, 128, 70
    g = gen(11)
    k, v = rows_of(g, (total, hkv, d), torch.bfloat16), rows_of(g, (total, hkv, d), torch.bfloat16)
    slots = torch.arange(total, dtype=torch.int32, device="cuda") + 20
    plain = new_cache(pages, hkv, page, d)
    if layout == "pages_rows_heads":
        base = [torch.zeros((pages, page, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
        codes = [x.transpose(1, 2).view(torch.float8_e4m3fn) for x in base]
        exps = [torch.full((hkv, pages, page), 127, dtype=torch.uint8, device="cuda").transpose(0, 1) for _ in range(2)]
    elif layout == "interleaved":
        base = torch.zeros((pages, 2, hkv, page, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        ebase = torch.full((pages, hkv, 2, page), 127, dtype=torch.uint8, device="cuda")
        codes, exps = [base[:, i] for i in range(2)], [ebase[:, :, i] for i in range(2)]
    else:   # codes and exponents of a page next to each other
        n = hkv * page
        base = torch.full((pages, 2 * n * (d + 1)), 127, dtype=torch.uint8, device="cuda")
        base[:, :2 * n * d] = 0
        codes = [base[:, i * n * d:(i + 1) * n * d].view(pages, hkv, page, d).view(torch.float8_e4m3fn) for i in range(2)]
        exps = [base[:, 2 * n * d + i * n:2 * n * d + (i + 1) * n].view(pages, hkv, page) for i in range(2)]
    cache = codes + exps
    for c in (plain, cache):
        fa2.fa2_paged_append_fp8(k, v, slots, *c)
    for a, b in zip(plain, cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for a, b in zip(fa2.fa2_paged_read_fp8(slots, *plain), fa2.fa2_paged_read_fp8(slots, *cache)):
        assert torch.equal(a, b)
    q = torch.randn((3, 6, d), generator=g, device="cuda").to(torch.bfloat16)
    table, cu, lens = i32([[2, 4, 3, 1, 5], [1, 2, 3, 4, 5]]), i32([0, 2, 3]), i32([70, 33])
    outs = [fa2.fa2_paged_fwd_fp8(q, *c, table, cu, lens, window_right=0) for c in (plain, cache)]
    assert status() == fa2.FA2_OK
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_rows_cut_from_a_projection_and_interleaved_outputs():
    g = gen(5)
    fused = rows_of(g, (33, 9, 64), torch.float16)   # [q | k | v] heads
    k, v = fused[:, 3:6], fused[:, 6:]
    slots = torch.arange(33, dtype=torch.int32, device="cuda")
    a, b = new_cache(5, 3, 8, 64), new_cache(5, 3, 8, 64)
    fa2.fa2_paged_append_fp8(k, v, slots, *a)
    fa2.fa2_paged_append_fp8(k.contiguous(), v.contiguous(), slots, *b)
    both = torch.zeros((33, 2, 3, 64), dtype=torch.float16, device="cuda")
    fa2.fa2_paged_read_fp8(slots, *a, k=both[:, 0], v=both[:, 1])
    want = fa2.fa2_paged_read_fp8(slots, *b, dtype=torch.float16)
    assert status() == fa2.FA2_OK
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(both[:, 0], want[0]) and torch.equal(both[:, 1], want[1])


def test_slots_past_the_cache_are_skipped_and_reported():
    g = gen(6)
    x = rows_of(g, (4, 2, 128), torch.bfloat16)
    cache = new_cache(2, 2, 8, 128)
    fa2.fa2_paged_append_fp8(x, x, i32([3, 16, -5, 15]), *cache)
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    out = [torch.full((4, 2, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa2.fa2_paged_read_fp8(i32([3, 1 << 30, 15, 3]), *cache, k=out[0], v=out[1])   # a slot may repeat
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    for y in out:
        assert (y[1] == 9).all() and torch.equal(y[0], y[3]) and not (y[2] == 9).any()
    used = cache[0].view(torch.uint8).reshape(2, 2, 8, 128).amax((1, 3)).reshape(-1)
    assert used.nonzero().flatten().tolist() == [3, 15]


# ---------------------------------------------------------------- attention

def seen_mask(n_q, n_k, wl, wr, pre, sinks=0):
    i = torch.arange(n_q, device="cuda")[:, None] + (n_k - n_q)
    j = torch.arange(n_k, device="cuda")[None, :]
    seen = torch.ones((n_q, n_k), dtype=torch.bool, device="cuda")
    edge = j <= i + wr if wr >= 0 else seen
    if wl >= 0:
        seen = seen & (j >= i - wl)
    return (seen & edge) | (j < pre) | ((j < sinks) & edge)


class Problem:
    """Random queries and an 8-bit cache of the given lengths, pages in random order; rows that no sequence holds are
    NaN codes with any exponent."""

    def __init__(self, lens_q, lens_k, hq, hkv, d, dtype, page, seed, sink=False):
        self.lens_q, self.lens_k, self.page, self.d, self.hq, self.hkv = list(lens_q), list(lens_k), page, d, hq, hkv
        g, dt = gen(seed), DT[dtype]
        need = [-(-n // page) for n in lens_k]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g, device="cuda")[:sum(need)].tolist()
        table = np.full((len(lens_k), max(need) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.q = torch.randn((max(1, sum(lens_q)), hq, d), generator=g, device="cuda").to(dt)
        self.cache = new_cache(pages, hkv, page, d, fill=0x7f)
        for x in self.cache[2:]:
            x.copy_(torch.randint(0, 256, x.shape, generator=g, device="cuda", dtype=torch.uint8))
        for b, n in enumerate(lens_k):
            if n == 0:
                continue
            k, v = rows_of(g, (n, hkv, d), dt), rows_of(g, (n, hkv, d), dt)
            if sink:   # the first key takes most of the weight, and its value is small
                k[0] = self.q[0].float().reshape(hkv, -1, d).mean(1).mul(4).to(dt)
                v[0] = v[0] * 2.0 ** -9
            j = torch.arange(n, device="cuda")
            slots = (self.table[b, j // page].long() * page + j % page).to(torch.int32)
            fa2.fa2_paged_append_fp8(k, v, slots, *self.cache)
        self.cu, self.lens = i32(np.concatenate([[0], np.cumsum(lens_q)])), i32(lens_k)

    def run(self, **kw):
        kw.setdefault("max_seqlen_q", max(1, max(self.lens_q)))
        return fa2.fa2_paged_fwd_fp8(self.q, *self.cache, self.table, self.cu, self.lens, **kw)

    def keys(self, b, i):
        """(codes, exponents) in float64 of sequence b, K (0) or V (1): [hkv, n, d], [hkv, n]."""
        j = torch.arange(self.lens_k[b], device="cuda")
        page_of, at = self.table[b, j // self.page].long(), j % self.page
        codes = self.cache[i].view(torch.uint8)[page_of, :, at].long()
        exps = self.cache[2 + i][page_of, :, at].double() - 127
        return torch.from_numpy(VALUES).cuda()[codes].transpose(0, 1), exps.T

    def check(self, o, lse, scale=None, window_left=-1, window_right=-1, prefix_len=0, sink_len=0, skip=(), u=None,
              e_max=None):
        d, group = self.d, self.hq // self.hkv
        scale = 1.0 / d ** 0.5 if scale is None else scale
        u = torch.finfo(o.dtype).eps / 2 if u is None else u
        row = 0
        for b, (n, n_k) in enumerate(zip(self.lens_q, self.lens_k)):
            if b in skip or n == 0:
                row += n
                continue
            (kc, ke), (vc, ve) = self.keys(b, 0), self.keys(b, 1)
            hidden = ~seen_mask(n, n_k, window_left, window_right, prefix_len, sink_len)
            kc, vc = (x.masked_fill(hidden.all(0)[None, :, None], 0.0) for x in (kc, vc))
            ke, ve = (x.masked_fill(hidden.all(0)[None], 0.0) for x in (ke, ve))
            k, v, unit, kc, vc = (x.repeat_interleave(group, 0) for x in (
                kc * torch.exp2(ke)[..., None], vc * torch.exp2(ve)[..., None], torch.exp2(ve), kc, vc))
            q = self.q[row:row + n].double().transpose(0, 1)
            s = (scale * q @ k.transpose(1, 2)).masked_fill(hidden, -np.inf)
            ref_l = torch.logsumexp(s, -1) if n_k else torch.full(s.shape[:2], -np.inf, device="cuda").double()
            empty = torch.isinf(ref_l)
            p = torch.exp(s - torch.where(empty, torch.zeros_like(ref_l), ref_l)[..., None])
            ref_o, a = p @ v, p @ v.abs()
            got_o, got_l = o[row:row + n].double().transpose(0, 1), lse[:, row:row + n].double()
            assert torch.equal(torch.isneginf(got_l), empty), "sequence %d: rows without keys" % b
            assert (got_o[empty] == 0).all(), "sequence %d: a row without keys is not zero" % b
            assert torch.isfinite(got_o).all(), "sequence %d: non-finite output" % b
            if n_k:
                size = (q.abs() @ k.abs().transpose(1, 2)).masked_fill(hidden, 0.0).amax(-1)
                lost = 2.0 ** -25 * q.abs().amax(-1) * (k.abs().sum(-1)[:, None].masked_fill(hidden, 0.0)).amax(-1)
                ds = abs(scale) * (1.07 * d * 2.0 ** -23 * size + lost)
                n_vis = (~hidden).sum(-1).double()[None, :]
                small = 2.0 ** -18 + 2.0 ** -23 * (ve.abs().max() if e_max is None else e_max)
                floor = 2.0 ** -22 * (p * unit[:, None]).amax(-1)[..., None] * ((~hidden).double() @ vc.abs())
                tol = u * ref_o.abs() + floor + 1e-7 + a * (
                    2.0 ** -12 + 2 * ds + 2 * n_vis * 2.0 ** -23 + small)[..., None]
                worst = ((got_o - ref_o).abs() / tol)[~empty]
                assert worst.numel() == 0 or worst.max() <= 1, "sequence %d: O off by %.2f tolerances" % (b, worst.max())
                tol = ds + n_vis * 2.0 ** -23 + small + 2.0 ** -22 * ref_l.abs()
                worst = ((got_l - ref_l).abs() / tol)[~empty]
                assert worst.numel() == 0 or worst.max() <= 1, "sequence %d: L off by %.2f tolerances" % (b, worst.max())
            row += n


def test_one_key_tile():
    """The smallest call: one sequence, one token, up to 128 keys, each head dim."""
    for d in (128, 256, 64):
        for n_k in (1, 64, 128, 130):
            p = Problem([1], [n_k], 2, 2, d, "bf16", 16, seed=n_k)
            o, lse = p.run(window_right=0)
            assert status() == fa2.FA2_OK
            p.check(o, lse, window_right=0)


BATCHES = {
    "decode": ([1] * 7, [1, 17, 64, 65, 700, 129, 4097]),
    "ragged": ([1, 0, 5, 130, 33, 1, 3, 64], [300, 40, 5, 131, 1000, 0, 2, 64]),
    "chunk": ([200, 1], [1500, 2500]),
}
MASKS = {"causal": dict(window_right=0), "full": dict(), "window": dict(window_left=100, window_right=0),
         "prefix": dict(window_left=70, window_right=0, prefix_len=4), "wide": dict(window_left=130, window_right=3, prefix_len=100),
         "sinks": dict(window_left=90, window_right=0, sink_len=70), "self": dict(window_left=0, window_right=0)}


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "fp16"), (64, "bf16"), (128, "fp16"),
                                     (256, "bf16")])
@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("batch", sorted(BATCHES))
def test_attention_against_definition(batch, mask, d, dtype):
    lens_q, lens_k = BATCHES[batch]
    page = {"decode": 16, "ragged": 8, "chunk": 64}[batch]
    group = {"decode": 4, "ragged": 3, "chunk": 1}[batch]
    p = Problem(lens_q, lens_k, 2 * group, 2, d, dtype, page, seed=d + len(batch))
    o, lse = p.run(**MASKS[mask])
    assert status() == fa2.FA2_OK
    p.check(o, lse, **MASKS[mask])


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 192, 1024])
@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 1), (5, 2), (7, 1), (9, 1), (16, 1), (17, 1), (33, 1), (37, 1), (128, 1)])
def test_page_sizes_and_groups(page, group, hkv):
    p = Problem([1, 9, 40, 1], [1025, 300, 40, 63], group * hkv, hkv, 128, "bf16", page, seed=page + group)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


@pytest.mark.parametrize("tokens,group", [(1, 8), (1, 9), (2, 8), (1, 16), (1, 17), (1, 32), (4, 8), (5, 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_a_tile(tokens, group, d):
    """8, 16 and 32 rows a tile, and past them, over enough keys that pairs are cut and merged."""
    p = Problem([tokens, 1, tokens], [3000, 777, 20000], group, 1, d, "fp16", 64, seed=tokens + group)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


@pytest.mark.parametrize("batch", [1, 32, 33, 300])
def test_batches(batch):
    r = np.random.RandomState(batch)
    p = Problem([int(x) for x in r.randint(0, 3, batch)], [int(x) for x in r.randint(2, 900, batch)], 8, 2, 128, "bf16", 16,
                seed=batch)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_sink_of_large_weight_and_small_values(d):
    """One key holds most of P, and its value is 2^-9 of the others': the others' P keeps its bits."""
    p = Problem([1, 3], [6000, 900], 4, 1, d, "bf16", 32, seed=d, sink=True)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


@pytest.mark.parametrize("low,high", [(-58, -50), (40, 52), (-60, 52)])
def test_exponents_far_from_zero(low, high):
    """Values whose rows' exponents lie near the ends, or far apart: L counts every key, O what its values weigh."""
    n, d = 700, 128
    p = Problem([1, 2], [n, 300], 4, 2, d, "bf16", 16, seed=17)
    g = gen(18)
    for b, m in ((0, n), (1, 300)):
        j = torch.arange(m, device="cuda")
        size = torch.randint(low, high + 1, (m, 2, 1), generator=g, device="cuda").float()
        k = torch.randn((m, 2, d), generator=g, device="cuda").bfloat16()
        v = (torch.randn((m, 2, d), generator=g, device="cuda") * torch.exp2(size + 6)).bfloat16()
        slots = (p.table[b, j // 16].long() * 16 + j % 16).to(torch.int32)
        fa2.fa2_paged_append_fp8(k, v, slots, *p.cache)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    # (relative to the output's size: the check's own floor of 1e-7 would hide values of 2^-50)
    unit = 2.0 ** -high
    p.cache[3] = (p.cache[3].int() - high).clamp(0, 254).to(torch.uint8)
    p.check((o.double() * unit).float(), lse, window_right=0, u=torch.finfo(torch.bfloat16).eps / 2, e_max=60)


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 1e-4])
def test_scales(scale):
    p = Problem([1, 20], [400, 300], 8, 2, 64, "fp16", 16, seed=9)
    o, lse = p.run(window_right=0, scale=scale)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0, scale=scale)


@pytest.mark.parametrize("mask", [dict(window_left=2 ** 31 - 1, window_right=2 ** 31 - 1),
                                  dict(window_left=2 ** 31 - 1, window_right=0, sink_len=2 ** 31 - 1),
                                  dict(window_left=5, window_right=0, prefix_len=2 ** 31 - 1),
                                  dict(window_left=0, window_right=2, sink_len=3)])
def test_widest_and_narrowest_masks(mask):
    p = Problem([9, 1, 40], [300, 77, 40], 6, 2, 64, "fp16", 16, seed=14)
    o, lse = p.run(**mask)
    assert status() == fa2.FA2_OK
    p.check(o, lse, **mask)


def test_rising_scores_raise_the_maximum_on_every_step():
    """Key j's score grows with j: by 12 powers of two a step of 128 keys, past the margin of 8, and by less."""
    for rise in (12.0, 7.9, 3.0):
        p = Problem([1], [2000], 2, 1, 128, "bf16", 16, seed=2)
        p.q.zero_()
        p.q[..., 0] = 1.0
        n, d = 2000, 128
        j = torch.arange(n, device="cuda")
        k = torch.zeros((n, 1, d), device="cuda")
        k[:, 0, 0] = j * rise / 128 * np.log(2.0) + 1.0
        v = torch.rand((n, 1, d), generator=gen(1), device="cuda") * 2 - 1
        slots = (p.table[0, j // 16].long() * 16 + j % 16).to(torch.int32)
        fa2.fa2_paged_append_fp8(k.bfloat16(), v.bfloat16(), slots, *p.cache)
        o, lse = p.run(window_right=0, scale=1.0)
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0, scale=1.0)


def test_reads_what_reading_back_and_the_16_bit_forward_give():
    """Append, read back into a 16-bit cache, and both forwards: one function of the same values."""
    lens_k, page = [700, 1024, 33], 16
    p = Problem([3, 1, 20], lens_k, 8, 2, 128, "bf16", page, seed=4)
    o, lse = p.run(window_right=0)
    pages = p.cache[0].shape[0]
    slots = torch.arange(pages * page, dtype=torch.int32, device="cuda")
    for x in p.cache[:2]:   # (rows no sequence holds read back as NaN; the forward does not see them)
        assert torch.isnan(x.float()).any()
    k, v = fa2.fa2_paged_read_fp8(slots, *p.cache)
    k16, v16 = (x.view(pages, page, 2, 128).transpose(1, 2) for x in (k, v))
    o16, lse16 = fa2.fa2_paged_fwd(p.q, k16, v16, p.table, p.cu, p.lens, window_right=0, max_seqlen_q=20)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)
    assert torch.allclose(lse, lse16, rtol=2e-5, atol=2e-5)
    # O: each side's own roundings of P and O to 16 bits, at |v| below 16
    assert (o.float() - o16.float()).abs().max() <= 16 * 3 * 2.0 ** -8


# ---------------------------------------------------------------- refusals on the device, streams, graphs

def test_bad_lengths_offsets_and_pages_are_reported():
    p = Problem([1, 2, 1], [300, 40, 500], 4, 2, 128, "bf16", 16, seed=8)
    o, lse = p.run(window_right=0)
    p.lens[1] = p.table.shape[1] * 16 + 1
    o2, lse2 = torch.full_like(o, 5.0), torch.full_like(lse, 5.0)
    p.run(window_right=0, o=o2, lse=lse2)
    assert status() == fa2.FA2_ERR_DEVICE_SEQLENS
    assert (o2[1:3] == 5).all() and (lse2[:, 1:3] == 5).all()
    p.lens[1] = 40
    p.check(o2, lse2, window_right=0, skip=(1,))
    kept = p.table[2, 3].item()
    for bad in (-1, p.cache[0].shape[0], 1 << 30):   # a page out of range: zero codes, exponent 0
        p.table[2, 3] = bad
        o3, lse3 = p.run(window_right=0)
        assert status() == fa2.FA2_ERR_DEVICE_PAGES
        p.table[2, 3] = kept
        saved = [x[kept].clone() for x in p.cache]
        p.cache[0].view(torch.uint8)[kept], p.cache[1].view(torch.uint8)[kept] = 0, 0
        p.cache[2][kept], p.cache[3][kept] = 127, 127
        p.check(o3, lse3, window_right=0)
        for x, y in zip(p.cache, saved):
            x.view(torch.uint8)[kept] = y.view(torch.uint8)
    assert status() == fa2.FA2_OK


def test_a_nan_makes_its_row_nan():
    p = Problem([2, 1], [300, 40], 4, 2, 128, "bf16", 16, seed=8)
    p.q[1, 3, 7] = float("nan")
    page, row = p.table[1, 1].item(), 3
    p.cache[0].view(torch.uint8)[page, 0, row, 5] = 0x7f   # a visible key of sequence 1, head 0
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    assert torch.isnan(o[1, 3]).all() and torch.isnan(lse[3, 1])
    assert torch.isnan(o[2, :2]).all() and torch.isnan(lse[:2, 2]).all()
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[1, :3]).all() and torch.isfinite(o[2, 2:]).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_an_infinity_in_a_query_row_makes_it_nan(dtype, value):
    p = Problem([3, 1], [300, 40], 4, 2, 64, dtype, 16, seed=9)
    p.q[1, 2, 60] = value
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    assert torch.isnan(o[1, 2]).all() and torch.isnan(lse[2, 1])
    o[1, 2], lse[2, 1] = 0, 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("d,mask", [(64, "causal"), (128, "window"), (256, "causal"), (128, "sinks")])
def test_more_pairs_than_ctas(d, mask):
    """Chunks whose pairs of query tile and head are several for each CTA, between decoding and idle requests."""
    p = Problem([700, 1, 0, 333, 5], [900, 500, 9, 333, 1200], 8, 8, d, "bf16", 32, seed=11)
    o, lse = p.run(**MASKS[mask])
    assert status() == fa2.FA2_OK
    p.check(o, lse, **MASKS[mask])


def test_rows_outside_sequences_are_left_and_runs_repeat():
    p = Problem([2, 0, 3], [77, 10, 2000], 4, 1, 128, "fp16", 16, seed=10)
    q = torch.cat([p.q, p.q[:3]])
    o, lse = torch.full_like(q, 3.0), torch.full((4, q.shape[0]), 3.0, device="cuda")
    fa2.fa2_paged_fwd_fp8(q, *p.cache, p.table, p.cu, p.lens, o=o, lse=lse, window_right=0, max_seqlen_q=3)
    assert (o[5:] == 3).all() and (lse[:, 5:] == 3).all()
    p.check(o[:5], lse[:, :5], window_right=0)
    again = fa2.fa2_paged_fwd_fp8(q, *p.cache, p.table, p.cu, p.lens, window_right=0, max_seqlen_q=3)
    assert torch.equal(again[0][:5], o[:5]) and torch.equal(again[1][:, :5], lse[:, :5])
    assert status() == fa2.FA2_OK


def test_a_serving_step_on_a_stream_and_in_a_graph():
    """Plan, append and attention of two steps, captured once and replayed with new lengths, as eager calls give."""
    page, hkv, d, hq = 16, 2, 128, 8
    g = gen(12)
    start = [40, 0, 300]
    steps = [[1, 50, 1], [1, 1, 2]]
    k0, v0 = rows_of(g, (340, hkv, d), torch.bfloat16), rows_of(g, (340, hkv, d), torch.bfloat16)
    total = 64
    inputs = [[rows_of(g, (total, h, d), torch.bfloat16) for h in (hq, hkv, hkv)] for _ in steps]

    def server():
        cache = new_cache(64, hkv, page, d)
        table = torch.full((3, 32), -1, dtype=torch.int32, device="cuda")
        table[0, :3], table[2, :19] = i32([60, 61, 62]), i32(list(range(40, 59)))
        j = torch.arange(300, device="cuda")
        fa2.fa2_paged_append_fp8(k0[:40], v0[:40], (table[0, j[:40] // page] * page + j[:40] % page).to(torch.int32), *cache)
        fa2.fa2_paged_append_fp8(k0[40:], v0[40:], (table[2, j // page] * page + j % page).to(torch.int32), *cache)
        return cache, table, i32(list(range(40))), i32([40])

    def step(cache, table, free, count, ctx, new, q, k, v):
        cu, lens, slots, left = fa2.fa2_paged_plan(ctx, new, table, free, count, 64, page, total)
        fa2.fa2_paged_append_fp8(k, v, slots, *cache)
        o, lse = fa2.fa2_paged_fwd_fp8(q, *cache, table, cu, lens, window_right=0, max_seqlen_q=total)
        return o, lse, lens, left

    want = []
    cache, table, free, count = server()
    ctx = i32(start)
    for new, x in zip(steps, inputs):
        o, lse, ctx, count = step(cache, table, free, count, ctx, i32(new), *x)
        want.append((o[:sum(new)].clone(), lse[:, :sum(new)].clone()))
    stream = torch.cuda.Stream()
    cache2, table2, free2, count2 = server()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        ctx2, new2, x2 = i32(start), i32(steps[0]), [t.clone() for t in inputs[0]]
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            o2, lse2, lens2, left2 = step(cache2, table2, free2, count2, ctx2, new2, *x2)
        for i, new in enumerate(steps):
            new2.copy_(i32(new))
            for a, b in zip(x2, inputs[i]):
                a.copy_(b)
            graph.replay()
            n = sum(new)
            assert torch.equal(o2[:n], want[i][0]) and torch.equal(lse2[:, :n], want[i][1])
            ctx2.copy_(lens2)
            count2.copy_(left2)
    assert status() == fa2.FA2_OK
    for a, b in zip(cache, cache2):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_calls_at_once_with_their_own_workspaces():
    p = Problem([1] * 5, [900, 3000, 20, 70, 4000], 8, 2, 128, "bf16", 16, seed=14)
    want = p.run(window_right=0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [p.run(window_right=0, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    need = fa2.fa2_paged_fwd_fp8_workspace_bytes(p.q, *p.cache, p.table, p.cu, p.lens, max_seqlen_q=1)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")   # written before it is read
    o, lse = p.run(window_right=0, workspace=ws)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert status() == fa2.FA2_OK


def test_long_cache_past_2_31_bytes():
    """Offsets past 2^32 bytes: pages at the end of a cache of 5 GB."""
    hkv, d, page = 4, 128, 64
    pages = (5 << 30) // (hkv * d * page)
    g = gen(15)
    cache = [torch.empty((pages, hkv, page, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    cache += [torch.full((pages, hkv, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    n = 1000
    table = (pages - 1 - torch.arange(16, device="cuda")).to(torch.int32)[None].contiguous()
    p = Problem([1], [n], 8, hkv, d, "bf16", page, seed=15)
    k, v = rows_of(g, (n, hkv, d), torch.bfloat16), rows_of(g, (n, hkv, d), torch.bfloat16)
    j = torch.arange(n, device="cuda")
    slots = (table[0, j // page] * page + j % page).to(torch.int32)
    fa2.fa2_paged_append_fp8(k, v, slots, *cache)
    back = fa2.fa2_paged_read_fp8(slots, *cache)
    small = new_cache(16, hkv, page, d)
    fa2.fa2_paged_append_fp8(k, v, j.to(torch.int32), *small)
    want = fa2.fa2_paged_read_fp8(j.to(torch.int32), *small)
    assert torch.equal(back[0], want[0]) and torch.equal(back[1], want[1])
    p.cache, p.table = cache, table
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


def test_binding_checks_types_and_shapes():
    cache = new_cache(4, 2, 16, 64)
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    slots = i32([0, 1, 2])
    with pytest.raises(TypeError):
        fa2.fa2_paged_append_fp8(x.float(), x.float(), slots, *cache)
    with pytest.raises(TypeError):
        fa2.fa2_paged_append_fp8(x, x, slots, cache[0].view(torch.uint8), *cache[1:])
    with pytest.raises(TypeError):
        fa2.fa2_paged_append_fp8(x, x, slots, *cache[:2], cache[2].to(torch.int8), cache[3])
    with pytest.raises(ValueError):
        fa2.fa2_paged_append_fp8(x, x, slots, *cache[:2], cache[2][:, :, :8], cache[3][:, :, :8])
    with pytest.raises(ValueError):
        fa2.fa2_paged_append_fp8(x[:, :1], x[:, :1], slots, *cache)
    with pytest.raises(ValueError):
        fa2.fa2_paged_read_fp8(slots.long(), *cache)
    with pytest.raises(TypeError):
        fa2.fa2_paged_read_fp8(slots, *cache, dtype=torch.float32)
    with pytest.raises(ValueError):
        fa2.fa2_paged_read_fp8(slots, *cache, k=x[:2], v=x[:2])
    with pytest.raises(fa2.Fa2Error):
        fa2.fa2_paged_read_fp8(slots, *cache, k=x, v=x)   # one place for both
    q, table, cu, lens = x.repeat(1, 2, 1), i32([[0, 1]]), i32([0, 1]), i32([3])
    with pytest.raises(TypeError):
        fa2.fa2_paged_fwd_fp8(q.float(), *cache, table, cu, lens)
    with pytest.raises(ValueError):
        fa2.fa2_paged_fwd_fp8(q[..., :32], *cache, table, cu, lens)
    with pytest.raises(fa2.Fa2Error):
        fa2.fa2_paged_fwd_fp8(q, *cache, table, cu, lens, window_left=-3)
    with pytest.raises(fa2.Fa2Error):
        fa2.fa2_paged_fwd_fp8(q, *cache, table, cu, lens, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    version = cache[0]._version
    fa2.fa2_paged_append_fp8(x, x, slots, *cache)
    assert cache[0]._version > version   # torch knows of the write
    assert status() == fa2.FA2_OK
