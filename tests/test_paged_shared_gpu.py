"""Attention of sequences that share the first pages of their prompts
(fa2_paged_fwd_shared) on the GPU, against the definition in 64 bits.

Each output is that of fa2_paged_fwd, whose tolerances (test_paged_gpu) hold: a
shared length only changes where a row's keys are cut into partial sums, and a
P rounded in either pass is rounded once.  Inputs, block tables and the check
are that module's; here the rows of a group begin with the same pages."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build
from test_paged_gpu import Problem, i32, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    fa2.load_library()
    yield
    code, detail = fa2.fa2_get_device_status()
    assert code == fa2.FA2_OK, "device status word set: 0x%x" % detail


class Shared(Problem):
    """groups: (sequences, shared keys) of each group, in order; the sequences of a group get its first whole pages
    (sequences past the last group share nothing).  Their own copies of those pages hold NaN."""

    def __init__(self, lens_q, lens_k, groups, *args, **kw):
        super().__init__(lens_q, lens_k, *args, **kw)
        cuts = np.cumsum([0] + [n for n, _ in groups])
        nan = []
        for g, (n, shared) in enumerate(groups):
            for b in range(cuts[g] + 1, cuts[g + 1]):
                common = shared // self.page
                nan += self.table[b, :common].tolist()
                self.table[b, :common] = self.table[cuts[g], :common]
        for c in (self.k, self.v):
            if nan:
                c[torch.tensor(nan, device="cuda")] = float("nan")
        self.cu_groups, self.shared = i32(cuts), i32([s for _, s in groups])

    def run(self, **kw):
        kw.setdefault("max_seqlen_q", max(1, max(self.lens_q)))
        kw.setdefault("window_right", 0)
        return fa2.fa2_paged_fwd_shared(self.q, self.k, self.v, self.table, self.cu, self.lens, self.cu_groups, self.shared,
                                        **kw)


def lens_of(groups, own, new):
    """Keys of sequences: their group's shared ones, `own` cached ones and the new tokens."""
    shared = [s for n, s in groups for _ in range(n)]
    shared += [0] * (len(own) - len(shared))
    return [s + o + n for s, o, n in zip(shared, own, new)]


# (groups, cached keys of their own, new tokens)
BATCHES = {
    "decode": ([(4, 1000)], [0, 1, 63, 700], [1, 1, 1, 1]),
    "groups": ([(3, 200), (1, 500), (2, 64), (3, 63)], [5, 0, 300, 40, 1, 2, 3, 4, 5, 900, 0], [1] * 11),
    "drafted": ([(2, 3000), (3, 129)], [1, 50, 0, 7, 1000], [5, 3, 1, 2, 4]),
    "chunks": ([(3, 700), (2, 320)], [0, 100, 3, 200, 1], [130, 1, 64, 33, 200]),
    "idle": ([(3, 500), (3, 260)], [9, 4, 100, 30, 0, 11], [0, 2, 1, 1, 0, 0]),
}


@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "fp16"), (64, "bf16"), (128, "fp16"),
                                     (256, "bf16")])
@pytest.mark.parametrize("right", [0, -1])
@pytest.mark.parametrize("batch", sorted(BATCHES))
def test_attention_against_definition(batch, right, d, dtype):
    groups, own, new = BATCHES[batch]
    page = {"decode": 16, "groups": 8, "drafted": 64, "chunks": 32, "idle": 16}[batch]
    group = {"decode": 4, "groups": 3, "drafted": 8, "chunks": 2, "idle": 1}[batch]
    p = Shared(new, lens_of(groups, own, new), groups, 2 * group, 2, d, dtype, page, seed=d + len(batch), fill=float("nan"))
    o, lse = p.run(window_right=right)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=right)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 192])
@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 1), (5, 2), (7, 1), (16, 1), (33, 1), (128, 1)])
def test_page_sizes_and_groups(page, group, hkv):
    groups, own, new = [(2, 777), (2, 385)], [30, 1, 500, 0], [1, 3, 1, 9]
    p = Shared(new, lens_of(groups, own, new), groups, group * hkv, hkv, 128, "bf16", page, seed=page + group,
               fill=float("inf"))
    o, lse = p.run()
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


@pytest.mark.parametrize("batch", [2, 32, 33, 130])
def test_batches(batch):
    """Many sequences of one group, and of random groups, over enough keys that pairs are cut."""
    r = np.random.RandomState(batch)
    new = [int(x) for x in r.randint(0, 3, batch)]
    own = [int(x) for x in r.randint(0, 200, batch)]
    for groups in ([(batch, 5000)], [(1, 70), (batch - 1, 1500)] if batch > 2 else [(2, 90)],
                   [(2, int(s)) for s in r.randint(0, 600, batch // 2)]):
        p = Shared(new, lens_of(groups, own, new), groups, 8, 2, 128, "bf16", 16, seed=batch)
        o, lse = p.run()
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0)


@pytest.mark.parametrize("batch,d,most", [(193, 64, 3), (500, 128, 2), (385, 256, 2), (260, 128, 20)])
def test_hundreds_of_sequences(batch, d, most):
    """Several sequences for each thread that sums them, in some and in many groups, with short and long own keys."""
    r = np.random.RandomState(batch)
    new = [int(x) for x in r.randint(0, most, batch)]
    own = [int(x) for x in np.where(r.rand(batch) < 0.1, r.randint(0, 700, batch), r.randint(0, 30, batch))]
    for groups in ([(batch - 3, 900)], [(5, int(s)) for s in r.randint(0, 300, batch // 5)]):
        p = Shared(new, lens_of(groups, own, new), groups, 6, 2, d, "bf16", 16, seed=batch)
        o, lse = p.run()
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0)


def test_a_long_prefix_and_many_rows():
    """The shared pass in several query tiles (of 128 rows) of one group, cut and whole."""
    for tokens, shared in ((2, 20000), (60, 700)):
        groups, new = [(12, shared)], [tokens] * 12
        p = Shared(new, lens_of(groups, [3] * 12, new), groups, 16, 4, 128, "bf16", 64, seed=tokens)
        o, lse = p.run()
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0)


@pytest.mark.parametrize("hkv,tokens,batch", [(1, 62, 5), (2, 3, 70), (1, 302, 1)])
def test_more_query_tiles_of_groups_than_ctas(hkv, tokens, batch):
    """128 query heads a K/V head: every token is a query tile, and the groups have more of them than there are CTAs."""
    groups, new = ([(batch, 200)] if batch > 1 else [(1, 200)]), [tokens] * batch
    p = Shared(new, lens_of(groups, [2] * batch, new), groups, 128 * hkv, hkv, 64, "bf16", 16, seed=tokens)
    o, lse = p.run()
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_groups_of_several_lengths(d):
    """Up to 32 groups are laid out by query tile, more as they fall on the line."""
    r = np.random.RandomState(d)
    for n in (5, 32, 33, 90):
        groups = [(int(r.randint(1, 4)), int(r.randint(0, 900))) for _ in range(n)]
        batch = sum(g for g, _ in groups)
        new = [int(x) for x in r.randint(0, 4, batch)]
        own = [int(x) for x in r.randint(0, 100, batch)]
        p = Shared(new, lens_of(groups, own, new), groups, 6, 2, d, "bf16", 32, seed=n)
        o, lse = p.run()
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0)


def test_equals_the_forward_that_shares_nothing():
    groups, new = [(6, 2000)], [1] * 6
    p = Shared(new, lens_of(groups, [10 * i for i in range(6)], new), groups, 8, 2, 128, "bf16", 16, seed=3)
    o, lse = p.run()
    plain = fa2.fa2_paged_fwd(p.q, p.k, p.v, p.table, p.cu, p.lens, window_right=0, max_seqlen_q=1)
    p.shared.zero_()   # nothing is shared
    alone = p.run()
    assert status() == fa2.FA2_OK
    for x, l in ((o, lse), plain, alone):
        p.check(x, l, window_right=0)


def test_shared_keys_are_read_through_the_first_sequence():
    """Only the first table row's entries of the shared pages are looked at."""
    groups, new = [(4, 512)], [0, 1, 1, 2]
    p = Shared(new, lens_of(groups, [1, 2, 30, 4], new), groups, 4, 1, 64, "fp16", 16, seed=4)
    want = p.run()
    p.check(*want, window_right=0)
    p.table[1:, :32] = 1 << 30
    got = p.run()
    assert status() == fa2.FA2_OK
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_out_of_range_groups_are_reported():
    groups, new = [(3, 300), (2, 128)], [1, 2, 1, 1, 1]
    p = Shared(new, lens_of(groups, [0, 40, 10, 5, 6], new), groups, 4, 2, 128, "bf16", 16, seed=5)
    want = p.run()
    p.check(*want, window_right=0)
    rows = {0: slice(0, 1), 1: slice(1, 3), 2: slice(3, 4), 3: slice(4, 5), 4: slice(5, 6)}

    def left(skip, o, lse, code=fa2.FA2_ERR_DEVICE_SEQLENS):
        assert status() == code
        for b in skip:
            assert (o[rows[b]] == 5).all() and (lse[:, rows[b]] == 5).all()
        p.check(o, lse, window_right=0, skip=skip)

    def run(**kw):
        o, lse = torch.full_like(p.q, 5.0), torch.full((4, p.q.shape[0]), 5.0, device="cuda")
        p.run(o=o, lse=lse, **kw)
        return o, lse

    good = p.shared.clone()
    for bad in (-1, 1 << 30, p.table.shape[1] * 16 + 64):   # a length no sequence can have
        p.shared[1] = bad
        left((3, 4), *run())
        p.shared.copy_(good)
    # reaches into the new tokens of one sequence: sequence 0 has 300 cached keys, sequence 2 has 310
    p.shared[0] = 320
    row = p.table[1].clone()
    p.table[1, :20] = p.table[0, :20].clamp(min=0)
    o, lse = run()
    assert status() == fa2.FA2_ERR_DEVICE_SEQLENS
    assert (o[0] == 5).all() and (o[3] == 5).all() and not (o[1:3] == 5).any()
    p.shared.copy_(good)
    groups_before = p.cu_groups.clone()
    p.table[1] = row
    for cuts in ([0, 3, 1 << 30], [-7, -5, -3], [2, 2, 1], [0, 9, 3]):   # not within the batch: shares nothing
        p.cu_groups.copy_(i32(cuts))
        o, lse = run()
        assert status() == fa2.FA2_OK
        p.check(o, lse, window_right=0)
    p.cu_groups.copy_(groups_before)
    p.lens[1] = 1 << 30
    o, lse = run()
    assert status() == fa2.FA2_ERR_DEVICE_SEQLENS
    assert (o[1:3] == 5).all() and torch.equal(o[3:], want[0][3:])


def test_a_page_out_of_range_is_reported():
    groups, new = [(2, 256)], [1, 1]
    p = Shared(new, lens_of(groups, [4, 9], new), groups, 4, 2, 128, "bf16", 16, seed=6)
    kept = p.table[0, 3].item()
    p.table[0, 3] = p.k.shape[0]
    o, lse = p.run()
    assert status() == fa2.FA2_ERR_DEVICE_PAGES
    p.table[:, 3] = kept
    p.k[kept], p.v[kept] = 0, 0
    p.check(o, lse, window_right=0)


def test_nan_in_a_shared_key_reaches_all_who_see_it():
    groups, new = [(3, 256)], [1, 1, 1]
    p = Shared(new, lens_of(groups, [4, 9, 200], new), groups, 4, 2, 128, "bf16", 16, seed=7)
    p.k[p.table[0, 2].item(), 1, 3, 5] = float("nan")
    p.q[2, 0, 1] = float("nan")
    o, lse = p.run()
    assert status() == fa2.FA2_OK
    assert torch.isnan(o[:, 2:]).all() and torch.isnan(lse[2:]).all()
    assert torch.isnan(o[2, 0]).all() and torch.isnan(lse[0, 2])
    assert torch.isfinite(o[:2, :2]).all() and torch.isfinite(o[2, 1]).all()


def test_rows_outside_sequences_are_left_and_strides_hold():
    groups, new = [(3, 1000)], [1, 2, 1]
    p = Shared(new, lens_of(groups, [4, 9, 200], new), groups, 4, 2, 128, "bf16", 16, seed=8)
    want = p.run()
    total = 4 + 3
    wide = torch.zeros((total, 12, 128), dtype=torch.bfloat16, device="cuda")
    wide[:4, 4:8] = p.q
    o, lse = torch.full((total, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 50), 3.0, device="cuda")
    cu = p.cu
    fa2.fa2_paged_fwd_shared(wide[:, 4:8], p.k, p.v, p.table, cu, p.lens, p.cu_groups, p.shared, o=o[:, 2:6],
                             lse=lse[:, :total], window_right=0, max_seqlen_q=2)
    assert status() == fa2.FA2_OK
    assert (o[4:] == 3).all() and (o[:, :2] == 3).all() and (o[:, 6:] == 3).all() and (lse[:, 4:] == 3).all()
    p.check(o[:4, 2:6], lse[:, :4], window_right=0)
    p.check(*want, window_right=0)


def test_captured_calls_replay_with_new_lengths_and_groups():
    groups, new = [(4, 900), (2, 300)], [1, 1, 1, 1, 1, 1]
    p = Shared(new, lens_of(groups, [4, 9, 200, 0, 3, 70], new), groups, 8, 2, 128, "bf16", 16, seed=9)
    first = p.run()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        o, lse = p.run()
        o2, lse2 = p.run()   # a second one behind it, with a workspace of its own
    graph.replay()
    torch.cuda.synchronize()
    for x, l in ((o, lse), (o2, lse2)):
        assert torch.equal(x, first[0]) and torch.equal(l, first[1])
    p.shared.copy_(i32([64, 0]))
    p.lens.sub_(i32([0, 3, 100, 0, 1, 20]))
    p.lens_k = p.lens.tolist()
    graph.replay()
    p.check(o, lse, window_right=0)
    p.cu_groups.copy_(i32([0, 2, 2]))
    graph.replay()
    p.check(o2, lse2, window_right=0)
    assert status() == fa2.FA2_OK


def test_calls_on_streams_and_between_other_kernels():
    """Runs repeat bit for bit on other streams, at once, behind the append that wrote their keys, and with workspaces
    that hold anything."""
    groups, new = [(8, 3000)], [1] * 8
    p = Shared(new, lens_of(groups, [30 * i for i in range(8)], new), groups, 8, 2, 128, "bf16", 16, seed=10)
    want = p.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [p.run(stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    need = fa2.fa2_paged_fwd_shared_workspace_bytes(p.q, p.k, p.v, p.table, p.cu, p.lens, p.cu_groups, p.shared, max_seqlen_q=1)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        got.append(p.run(workspace=ws))
    # the last tokens' rows, appended right before the call
    at = torch.tensor([n - 1 for n in p.lens_k], device="cuda")
    page_of = p.table[torch.arange(8, device="cuda"), at // 16].long()
    slots = (page_of * 16 + at % 16).to(torch.int32)
    k, v = p.k[page_of, :, at % 16].clone(), p.v[page_of, :, at % 16].clone()
    for _ in range(5):
        p.k[page_of, :, at % 16] = 0
        fa2.fa2_paged_append(k, v, slots, p.k, p.v)
        got.append(p.run())
    torch.cuda.synchronize()
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(fa2.Fa2Error):
        p.run(workspace=ws[:need - 256])
    assert status() == fa2.FA2_OK


def test_a_serving_step_with_a_shared_prompt():
    """A prompt computed once, then requests that start from its pages: plan, append, shared attention, as separate
    copies of the prompt give."""
    page, hkv, hq, d, prompt, batch = 16, 2, 8, 128, 200, 4
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    kp, vp = rnd(prompt, hkv, d), rnd(prompt, hkv, d)
    whole = prompt // page                      # pages that can be shared
    cache = [torch.zeros((200, hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.full((batch, 40), -1, dtype=torch.int32, device="cuda")
    table[:, :whole] = torch.arange(whole, dtype=torch.int32, device="cuda")
    fa2.fa2_paged_append(kp[:whole * page], vp[:whole * page], torch.arange(whole * page, dtype=torch.int32, device="cuda"),
                         *cache)
    ctx, free, count = i32([whole * page] * batch), torch.arange(whole, 200, dtype=torch.int32, device="cuda"), i32([200 - whole])
    separate = [torch.zeros_like(x) for x in cache]
    table2 = torch.full_like(table, -1)
    for b in range(batch):
        table2[b, :whole] = torch.arange(whole, dtype=torch.int32, device="cuda") + 20 * b
        slots = torch.arange(whole * page, dtype=torch.int32, device="cuda") + 20 * b * page
        fa2.fa2_paged_append(kp[:whole * page], vp[:whole * page], slots, *separate)
    ctx2, free2, count2 = ctx.clone(), torch.arange(100, 200, dtype=torch.int32, device="cuda"), i32([100])
    groups, shared = i32([0, batch]), i32([whole * page])
    for new in ([30, 1, 8, 17], [1, 1, 1, 1], [1, 0, 2, 1]):
        total = sum(new)
        q, k, v = rnd(total, hq, d), rnd(total, hkv, d), rnd(total, hkv, d)
        cu, lens, slots, count = fa2.fa2_paged_plan(ctx, i32(new), table, free, count, 200, page, total)
        fa2.fa2_paged_append(k, v, slots, *cache)
        o, lse = fa2.fa2_paged_fwd_shared(q, *cache, table, cu, lens, groups, shared, window_right=0, max_seqlen_q=max(new))
        cu2, lens2, slots2, count2 = fa2.fa2_paged_plan(ctx2, i32(new), table2, free2, count2, 200, page, total)
        fa2.fa2_paged_append(k, v, slots2, *separate)
        o2, lse2 = fa2.fa2_paged_fwd(q, *separate, table2, cu2, lens2, window_right=0, max_seqlen_q=max(new))
        assert torch.allclose(lse, lse2, rtol=2e-5, atol=2e-5)
        # each side rounds P and O to 16 bits once: |v| below 8
        assert (o.float() - o2.float()).abs().max() <= 8 * 3 * 2.0 ** -8
        ctx, ctx2 = lens, lens2
    assert status() == fa2.FA2_OK
