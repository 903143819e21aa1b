"""Paged-cache entry points without a GPU: every refusal the C ABI and the
binding document happens before any CUDA call, and the workspace sizes follow
from the shapes alone.  Pointer values are stand-ins that are never
dereferenced: each call fails an argument check first."""
import ctypes

import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build

A = 0x100000
INVALID, UNSUPPORTED, MISALIGNED = fa2.FA2_ERR_INVALID_ARG, fa2.FA2_ERR_UNSUPPORTED, fa2.FA2_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    fa2_build.build()
    return fa2.load_library()


def _set(struct, **kw):
    for key, val in kw.items():
        target = struct.cache if not hasattr(struct, key) else struct
        if isinstance(val, list):
            getattr(target, key)[:] = val
        else:
            setattr(target, key, val)
    return struct


def _cache(c):
    # 4 pages of 16 rows, 2 heads, d = 64: 16 KB each
    c.k, c.v = 10 * A, 11 * A
    c.num_pages, c.page_size, c.heads, c.head_dim, c.dtype = 4, 16, 2, 64, 0
    c.k_strides[:] = [2048, 1024, 64]
    c.v_strides[:] = [2048, 1024, 64]


def _fwd(**kw):
    p = fa2.Fa2PagedParams()
    _cache(p.cache)
    p.q, p.o, p.lse, p.block_table, p.cu_seqlens_q, p.seqlens_k = A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A
    p.table_stride, p.lse_stride = 8, 5
    p.q_strides[:] = [256, 64]
    p.o_strides[:] = [256, 64]
    p.batch, p.heads, p.total_q, p.max_seqlen_q, p.max_pages = 3, 4, 5, 2, 8
    p.window_left, p.window_right, p.prefix_len, p.scale = -1, 0, 0, 0.125
    # `heads` exists in both structs: kv_heads names the cache's
    kv = kw.pop("kv_heads", None)
    if kv is not None:
        p.cache.heads = kv
    for key in ("k", "v"):
        if key in kw:
            setattr(p.cache, key, kw.pop(key))
    return _set(p, **kw)


def _call_fwd(lib, ws=20 * A, ws_bytes=None, **kw):
    p = _fwd(**kw)
    need = lib.fa2_paged_fwd_workspace_bytes(ctypes.byref(_fwd()))
    return lib.fa2_paged_fwd(ctypes.byref(p), ws, need if ws_bytes is None else ws_bytes, None)


def test_layout_matches_library(lib):
    assert lib.fa2_paged_params_size() == ctypes.sizeof(fa2.Fa2PagedParams)
    assert "paged" in fa2.fa2_status_string(fa2.FA2_ERR_DEVICE_PAGES)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(heads=0), INVALID), (dict(total_q=0), INVALID), (dict(max_seqlen_q=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(kv_heads=0), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(dtype=2), INVALID), (dict(heads=5), INVALID),                      # not a multiple of the K/V heads
    (dict(kv_heads=1, heads=129, lse_stride=5), UNSUPPORTED),                # group above 128
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=12), UNSUPPORTED), (dict(page_size=1), UNSUPPORTED),
    (dict(page_size=96), UNSUPPORTED), (dict(num_pages=1 << 28), UNSUPPORTED), (dict(max_pages=1 << 28), UNSUPPORTED),
    (dict(window_left=-2), INVALID), (dict(window_right=-2), INVALID), (dict(prefix_len=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=0), INVALID), (dict(o=0), INVALID), (dict(lse=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(block_table=0), INVALID), (dict(cu_seqlens_q=0), INVALID), (dict(seqlens_k=0), INVALID), (dict(ws=0), INVALID),
    (dict(q=A + 8), MISALIGNED), (dict(o=2 * A + 8), MISALIGNED), (dict(k=10 * A + 8), MISALIGNED),
    (dict(lse=3 * A + 2), MISALIGNED), (dict(block_table=4 * A + 2), MISALIGNED), (dict(cu_seqlens_q=5 * A + 1), MISALIGNED),
    (dict(seqlens_k=6 * A + 2), MISALIGNED), (dict(ws=20 * A + 16), MISALIGNED),
    (dict(q_strides=[260, 64]), MISALIGNED), (dict(o_strides=[256, 4]), MISALIGNED), (dict(k_strides=[2048, 1024, 68]), MISALIGNED),
    (dict(v_strides=[2048, 0, 64]), INVALID), (dict(q_strides=[-256, 64]), INVALID), (dict(o_strides=[1 << 40, 64]), INVALID),
    (dict(table_stride=-1), INVALID), (dict(lse_stride=4), INVALID), (dict(ws_bytes=0), INVALID),
    (dict(o=A + 64), INVALID), (dict(o=10 * A + 1024), INVALID), (dict(lse=2 * A + 64), INVALID),
    (dict(o=4 * A), INVALID), (dict(lse=5 * A), INVALID), (dict(lse=6 * A + 8), INVALID), (dict(ws=11 * A), INVALID),
])
def test_fwd_refusals(lib, kw, code):
    assert _call_fwd(lib, **kw) == code
    assert lib.fa2_paged_fwd(None, 20 * A, 1 << 30, None) == INVALID


def test_fwd_workspace_follows_shapes(lib):
    size = lambda **kw: lib.fa2_paged_fwd_workspace_bytes(ctypes.byref(_fwd(**kw)))
    # two partial states for each of 304 CTAs (152 at head dim 256): 2 x 2 rows (tokens x heads of a K/V head), d + 2
    # floats each, and 32 bytes per CTA for the merge, each part rounded up to 256 bytes
    assert size() == 608 * 4 * 64 * 4 + 608 * 4 * 2 * 4 + 9728
    assert size(head_dim=256) == 304 * 4 * 256 * 4 + 304 * 4 * 2 * 4 + 4864
    assert size(heads=5) == 0 and size(head_dim=80) == 0 and size(total_q=0) == 0
    assert lib.fa2_paged_fwd_workspace_bytes(None) == 0
    # bounded whatever the batch holds: 128 rows
    assert size(total_q=1 << 20, max_seqlen_q=1 << 20, batch=64) == 608 * 128 * 64 * 4 + 608 * 128 * 2 * 4 + 9728


def _append(**kw):
    p = fa2.Fa2PagedAppendParams()
    _cache(p.cache)
    p.k, p.v, p.slots, p.total = A, 2 * A, 3 * A, 5
    p.k_strides[:] = [128, 64]
    p.v_strides[:] = [128, 64]
    for key in ("cache_k", "cache_v", "cache_k_strides"):
        if key in kw:
            val = kw.pop(key)
            if isinstance(val, list):
                getattr(p.cache, key[6:])[:] = val
            else:
                setattr(p.cache, key[6:], val)
    return _set(p, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(total=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(slots=0), INVALID),
    (dict(cache_k=0), INVALID), (dict(heads=0), INVALID), (dict(dtype=7), INVALID), (dict(head_dim=32), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED), (dict(heads=65537), UNSUPPORTED),
    (dict(k=A + 8), MISALIGNED), (dict(v=2 * A + 4), MISALIGNED), (dict(slots=3 * A + 2), MISALIGNED),
    (dict(cache_v=11 * A + 8), MISALIGNED), (dict(k_strides=[132, 64]), MISALIGNED), (dict(v_strides=[128, -64]), INVALID),
    (dict(cache_k_strides=[2048, 1024, 4]), MISALIGNED),
    (dict(cache_v=10 * A), INVALID),                                          # k and v at one place
    (dict(k=10 * A + 2048), INVALID), (dict(slots=11 * A + 512), INVALID),    # inputs inside the cache
])
def test_append_refusals(lib, kw, code):
    assert lib.fa2_paged_append(ctypes.byref(_append(**kw)), None) == code
    assert lib.fa2_paged_append(None, None) == INVALID


def _plan(**kw):
    p = fa2.Fa2PagedPlanParams()
    names = ("context_lens", "query_lens", "free_pages", "free_count", "block_table", "cu_seqlens_q", "seqlens_k",
             "slots", "free_left")
    for i, name in enumerate(names):
        setattr(p, name, (i + 1) * A)
    p.table_stride, p.batch, p.max_pages, p.num_pages, p.page_size, p.total_q, p.num_free = 8, 3, 8, 64, 16, 10, 32
    return _set(p, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
    (dict(total_q=0), INVALID), (dict(num_free=-1), INVALID), (dict(batch=16385), UNSUPPORTED),
    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(max_pages=1 << 27, table_stride=1 << 27), UNSUPPORTED),
    (dict(table_stride=7), INVALID), (dict(context_lens=0), INVALID), (dict(query_lens=0), INVALID),
    (dict(free_pages=0), INVALID), (dict(free_count=0), INVALID), (dict(block_table=0), INVALID),
    (dict(cu_seqlens_q=0), INVALID), (dict(seqlens_k=0), INVALID), (dict(slots=0), INVALID), (dict(free_left=0), INVALID),
    (dict(slots=8 * A + 1), MISALIGNED), (dict(free_pages=3 * A + 2), MISALIGNED),
    (dict(free_left=4 * A), INVALID),            # the count cannot be updated in place
    (dict(seqlens_k=A), INVALID),                # nor the context lengths
    (dict(slots=5 * A + 32), INVALID), (dict(cu_seqlens_q=7 * A + 8), INVALID),
])
def test_plan_refusals(lib, kw, code):
    assert lib.fa2_paged_plan(ctypes.byref(_plan(**kw)), None) == code
    assert lib.fa2_paged_plan(None, None) == INVALID


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    cache = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    q = torch.zeros((5, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        fa2.fa2_paged_fwd(q, cache, cache.clone(), i32(3, 8), i32(4), i32(3))
    with pytest.raises(ValueError):
        fa2.fa2_paged_append(q[:, :2], q[:, 2:], i32(5), cache, cache.clone())
    with pytest.raises(ValueError):
        fa2.fa2_paged_plan(i32(3), i32(3), i32(3, 8), i32(4), i32(1), 4, 16, 5)
    with pytest.raises(TypeError):
        fa2.fa2_paged_append(q, None, i32(5), cache, cache.clone())
    with pytest.raises(TypeError):
        fa2.fa2_paged_plan([1, 2], i32(3), i32(3, 8), i32(4), i32(1), 4, 16, 5)
    with pytest.raises(ValueError):
        fa2.fa2_paged_fwd_workspace_bytes(q, cache, cache.clone(), i32(3, 8), i32(4), i32(3))
