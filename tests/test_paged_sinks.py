"""Sink keys of the paged forward (sink_len): the first keys of a sequence stay
visible to later queries beside a sliding window, and to none before them.

The definition, in 64 bits, and the tolerances are those of test_paged_gpu."""
import ctypes

import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build
import test_paged_cpu as cpu
import test_paged_gpu as paged

prefix_mask = paged.seen_mask


@pytest.fixture(scope="module")
def lib():
    fa2_build.build()
    return fa2.load_library()


@pytest.fixture
def gpu(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    code, detail = fa2.fa2_get_device_status()
    assert code == fa2.FA2_OK, "device status word set: 0x%x" % detail


def check(monkeypatch, p, o, lse, sinks, **kw):
    """Every output against the definition: band, prefix, or one of the first `sinks` keys up to the band's end."""
    def seen_mask(n_q, n_k, wl, wr, pre):
        i = torch.arange(n_q, device="cuda")[:, None] + (n_k - n_q)
        j = torch.arange(n_k, device="cuda")[None, :]
        end = i + wr if wr >= 0 else torch.full_like(i, n_k)
        return prefix_mask(n_q, n_k, wl, wr, pre) | ((j < sinks) & (j <= end))
    monkeypatch.setattr(paged, "seen_mask", seen_mask)
    p.check(o, lse, **kw)
    monkeypatch.setattr(paged, "seen_mask", prefix_mask)


def test_refusals(lib):
    assert cpu._call_fwd(lib, sink_len=-1) == fa2.FA2_ERR_INVALID_ARG
    assert lib.fa2_paged_fwd_workspace_bytes(ctypes.byref(cpu._fwd(sink_len=4))) == \
        lib.fa2_paged_fwd_workspace_bytes(ctypes.byref(cpu._fwd()))


@pytest.mark.gpu
def test_first_tokens_of_a_prompt_do_not_see_ahead(gpu):
    """Five tokens on an empty context beside four sinks: row i sees keys 0 .. i, as it does without a window."""
    p = paged.Problem([5], [5], 4, 2, 64, "fp16", 16, seed=1)
    o, lse = p.run(window_left=2, window_right=0, sink_len=4)
    causal, causal_l = p.run(window_right=0)
    assert torch.equal(o, causal) and torch.equal(lse, causal_l)
    p.check(o, lse, window_right=0)


# (new tokens, keys): prompts from their start, chunks after little and much context, decoding, more tokens than keys
BATCHES = {
    "prompts": ([5, 1, 130, 3, 64, 333], [5, 1, 130, 3, 64, 333], 3),
    "few": ([5, 1, 8, 3, 7, 2], [5, 1, 100, 1500, 4, 70], 4),
    "chunks": ([100, 0, 260, 1], [101, 7, 700, 3000], 1),
    "ahead": ([9, 200, 5], [4, 70, 0], 2),
    "decode": ([1] * 40, [1 + 37 * b for b in range(40)], 8),
}
MASKS = {"four": (70, 0, 4, 0), "window shorter": (3, 0, 100, 0), "right": (40, 2, 70, 0), "itself": (0, 0, 1, 0),
         "prefix too": (30, 0, 130, 65), "all": (10, 0, 10 ** 9, 0), "no right edge": (25, -1, 90, 0)}


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (256, "bf16")])
@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("batch", sorted(BATCHES))
def test_against_definition(gpu, monkeypatch, batch, mask, d, dtype):
    lens_q, lens_k, group = BATCHES[batch]
    wl, wr, sinks, pre = MASKS[mask]
    p = paged.Problem(lens_q, lens_k, 2 * group, 2, d, dtype, 16, seed=d + len(mask), fill=float("nan"))
    kw = dict(window_left=wl, window_right=wr, prefix_len=pre)
    o, lse = p.run(sink_len=sinks, **kw)
    assert paged.status() == fa2.FA2_OK
    check(monkeypatch, p, o, lse, sinks, **kw)


@pytest.mark.gpu
def test_equals_a_prefix_behind_the_sinks_and_nothing_without_a_window(gpu):
    p = paged.Problem([3, 1, 200], [400, 33, 900], 8, 2, 128, "bf16", 16, seed=7)
    for kw, other in ((dict(window_left=90, window_right=0), dict(prefix_len=4)), (dict(window_right=0), dict())):
        o, lse = p.run(sink_len=4, **kw)
        want, want_l = p.run(**other, **kw)
        assert torch.equal(o, want) and torch.equal(lse, want_l)


@pytest.mark.gpu
def test_long_prompt_in_chunks_equals_one_call(gpu, monkeypatch):
    """A prompt served in chunks: every chunk's rows as the definition over the whole prompt has them."""
    n, sinks, kw = 2000, 4, dict(window_left=255, window_right=0)
    whole = paged.Problem([n], [n], 8, 2, 128, "bf16", 64, seed=8)
    at = 0
    for m in (2, 1, 700, 64, 1, 1232):
        p = paged.Problem.__new__(paged.Problem)
        p.__dict__.update(whole.__dict__)
        p.lens_q, p.lens_k = [m], [at + m]
        p.q, p.cu, p.lens = whole.q[at:at + m], paged.i32([0, m]), paged.i32([at + m])
        o, lse = p.run(sink_len=sinks, **kw)
        check(monkeypatch, p, o, lse, sinks, **kw)
        at += m
    assert at == n


@pytest.mark.gpu
def test_on_a_stream_of_its_own(gpu, monkeypatch):
    p = paged.Problem([40, 1], [60, 300], 8, 2, 128, "bf16", 16, seed=9, fill=float("nan"))
    kw = dict(window_left=20, window_right=0)
    torch.cuda.synchronize()
    o, lse = p.run(sink_len=6, stream=torch.cuda.Stream(), **kw)
    assert paged.status() == fa2.FA2_OK
    check(monkeypatch, p, o, lse, 6, **kw)
