"""Entry points of the 8-bit paged cache without a GPU: every refusal the C ABI
and the binding document happens before any CUDA call, and workspace sizes
follow from the shapes alone.  Pointer values are stand-ins that are never
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


def _fill(struct, defaults, kw):
    """Sets fields; names that begin with cache_ are the cache's."""
    for key, val in {**defaults, **kw}.items():
        target, name = (struct.cache, key[6:]) if key.startswith("cache_") else (struct, key)
        if isinstance(val, list):
            getattr(target, name)[:] = val
        else:
            setattr(target, name, val)
    return struct


# 4 pages of 16 rows, 2 heads, d = 64: 8 KB of codes, 128 bytes of exponents
CACHE = dict(cache_k=10 * A, cache_v=11 * A, cache_k_exps=12 * A, cache_v_exps=13 * A, cache_k_strides=[2048, 1024, 64],
             cache_v_strides=[2048, 1024, 64], cache_k_exp_strides=[32, 16], cache_v_exp_strides=[32, 16],
             cache_num_pages=4, cache_page_size=16, cache_heads=2, cache_head_dim=64)


def _rows(**kw):
    return _fill(fa2.Fa2PagedRowsFp8Params(), dict(CACHE, k=A, v=2 * A, slots=3 * A, k_strides=[128, 64],
                                                   v_strides=[128, 64], total=5, dtype=0), kw)


CACHE_REFUSALS = [
    (dict(cache_k=0), INVALID), (dict(cache_v=0), INVALID), (dict(cache_k_exps=0), INVALID), (dict(cache_v_exps=0), INVALID),
    (dict(cache_heads=0), INVALID), (dict(cache_num_pages=0), INVALID), (dict(cache_page_size=0), INVALID),
    (dict(cache_head_dim=96), UNSUPPORTED), (dict(cache_page_size=24), UNSUPPORTED), (dict(cache_page_size=4), UNSUPPORTED),
    (dict(cache_num_pages=1 << 28), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
    (dict(cache_k=10 * A + 8), MISALIGNED), (dict(cache_v_exps=13 * A + 4), MISALIGNED),
    (dict(cache_k_strides=[2048, 1024, 72]), MISALIGNED), (dict(cache_v_strides=[2048, -1024, 64]), INVALID),
    (dict(cache_k_exp_strides=[36, 16]), MISALIGNED), (dict(cache_v_exp_strides=[0, 16]), INVALID),
    (dict(cache_k_exp_strides=[1 << 40, 16]), INVALID),
]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(total=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(slots=0), INVALID),
    (dict(cache_heads=65537), UNSUPPORTED), (dict(k=A + 8), MISALIGNED), (dict(slots=3 * A + 2), MISALIGNED),
    (dict(k_strides=[132, 64]), MISALIGNED), (dict(v_strides=[128, 0]), INVALID),
    (dict(k=10 * A + 4096), INVALID), (dict(v=13 * A), INVALID),              # rows inside the cache
])
def test_rows_refusals(lib, kw, code):
    assert lib.fa2_paged_append_fp8(ctypes.byref(_rows(**kw)), None) == code
    assert lib.fa2_paged_read_fp8(ctypes.byref(_rows(**kw)), None) == code


def test_what_is_written_overlaps_nothing(lib):
    append = lambda **kw: lib.fa2_paged_append_fp8(ctypes.byref(_rows(**kw)), None)
    read = lambda **kw: lib.fa2_paged_read_fp8(ctypes.byref(_rows(**kw)), None)
    assert append(cache_v=10 * A) == INVALID and append(cache_v_exps=12 * A) == INVALID
    assert append(cache_k_exps=11 * A) == INVALID and append(slots=11 * A + 64) == INVALID
    assert append(slots=12 * A + 8) == INVALID
    assert read(v=A) == INVALID and read(slots=2 * A + 64) == INVALID
    assert lib.fa2_paged_append_fp8(None, None) == INVALID and lib.fa2_paged_read_fp8(None, None) == INVALID


def _fwd(**kw):
    return _fill(fa2.Fa2PagedFp8Params(), dict(
        CACHE, q=A, o=2 * A, lse=3 * A, block_table=4 * A, cu_seqlens_q=5 * A, seqlens_k=6 * A, table_stride=8, lse_stride=5,
        q_strides=[256, 64], o_strides=[256, 64], batch=3, heads=4, total_q=5, max_seqlen_q=2, max_pages=8, window_left=-1,
        window_right=0, prefix_len=0, scale=0.125, sink_len=0, dtype=1), kw)


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS + [
    (dict(batch=0), INVALID), (dict(heads=0), INVALID), (dict(total_q=0), INVALID), (dict(max_seqlen_q=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(heads=5), INVALID), (dict(cache_heads=1, heads=129), UNSUPPORTED),
    (dict(max_pages=1 << 28), UNSUPPORTED), (dict(window_left=-2), INVALID), (dict(window_right=-2), INVALID),
    (dict(prefix_len=-1), INVALID), (dict(sink_len=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=0), INVALID), (dict(o=0), INVALID), (dict(lse=0), INVALID),
    (dict(block_table=0), INVALID), (dict(cu_seqlens_q=0), INVALID), (dict(seqlens_k=0), INVALID), (dict(ws=0), INVALID),
    (dict(q=A + 8), MISALIGNED), (dict(o=2 * A + 8), MISALIGNED), (dict(lse=3 * A + 2), MISALIGNED),
    (dict(ws=20 * A + 128), MISALIGNED), (dict(q_strides=[260, 64]), MISALIGNED), (dict(o_strides=[256, 4]), MISALIGNED),
    (dict(q_strides=[-256, 64]), INVALID), (dict(table_stride=-1), INVALID), (dict(lse_stride=4), INVALID),
    (dict(ws_bytes=0), INVALID), (dict(o=A + 64), INVALID), (dict(o=10 * A), INVALID), (dict(o=12 * A), INVALID),
    (dict(lse=13 * A + 64), INVALID), (dict(ws=11 * A), INVALID), (dict(o=4 * A), INVALID), (dict(lse=2 * A), INVALID),
])
def test_fwd_refusals(lib, kw, code):
    ws, ws_bytes = kw.pop("ws", 20 * A), kw.pop("ws_bytes", 1 << 24)
    assert lib.fa2_paged_fwd_fp8(ctypes.byref(_fwd(**kw)), ws, ws_bytes, None) == code
    assert lib.fa2_paged_fwd_fp8(None, ws, ws_bytes, None) == INVALID


def test_fwd_workspace_follows_shapes(lib):
    size = lambda **kw: lib.fa2_paged_fwd_fp8_workspace_bytes(ctypes.byref(_fwd(**kw)))
    assert lib.fa2_paged_fp8_params_size() == ctypes.sizeof(fa2.Fa2PagedFp8Params)
    # two partial states for each of 304 CTAs (152 at head dim 256 and with more than 16 rows a tile), as fa2_paged_fwd
    assert size() == 608 * 4 * 64 * 4 + 608 * 4 * 2 * 4 + 9728
    assert size(cache_head_dim=256) == 304 * 4 * 256 * 4 + 304 * 4 * 2 * 4 + 4864
    assert size(heads=5) == 0 and size(cache_head_dim=80) == 0 and size(total_q=0) == 0
    assert lib.fa2_paged_fwd_fp8_workspace_bytes(None) == 0
    # bounded whatever the batch holds: 32 rows
    assert size(total_q=1 << 20, max_seqlen_q=1 << 20, batch=64) == 304 * 32 * 64 * 4 + 304 * 32 * 2 * 4 + 4864


def test_binding_refuses_host_tensors(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    codes = [torch.zeros((4, 2, 16, 64), dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2)]
    exps = [torch.zeros((4, 2, 16), dtype=torch.uint8) for _ in range(2)]
    q = torch.zeros((5, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        fa2.fa2_paged_fwd_fp8(q, *codes, *exps, i32(3, 8), i32(4), i32(3))
    with pytest.raises(ValueError):
        fa2.fa2_paged_append_fp8(q[:, :2], q[:, 2:], i32(5), *codes, *exps)
    with pytest.raises(ValueError):
        fa2.fa2_paged_read_fp8(i32(5), *codes, *exps)
    with pytest.raises(TypeError):
        fa2.fa2_paged_append_fp8(q, None, i32(5), *codes, *exps)
    with pytest.raises(ValueError):
        fa2.fa2_paged_fwd_fp8_workspace_bytes(q, *codes, *exps, i32(3, 8), i32(4), i32(3))
