"""fa2_paged_fwd_shared without a GPU: its refusals happen before any CUDA call,
and its workspace follows from the shapes alone.  Pointer values are stand-ins
that are never dereferenced."""
import ctypes

import pytest
import torch

import exact_tiled_attention_fa2_gb300 as fa2
from exact_tiled_attention_fa2_gb300 import build as fa2_build

A = 0x10000000
INVALID, UNSUPPORTED, MISALIGNED = fa2.FA2_ERR_INVALID_ARG, fa2.FA2_ERR_UNSUPPORTED, fa2.FA2_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    fa2_build.build()
    return fa2.load_library()


def _params(**kw):
    p = fa2.Fa2PagedSharedParams()
    f, c = p.fwd, p.fwd.cache
    c.k, c.v = 10 * A, 11 * A
    c.num_pages, c.page_size, c.heads, c.head_dim, c.dtype = 4, 16, 2, 64, 0
    c.k_strides[:] = [2048, 1024, 64]
    c.v_strides[:] = [2048, 1024, 64]
    f.q, f.o, f.lse, f.block_table, f.cu_seqlens_q, f.seqlens_k = A, 2 * A, 3 * A, 4 * A, 5 * A, 6 * A
    f.table_stride, f.lse_stride = 8, 5
    f.q_strides[:] = [256, 64]
    f.o_strides[:] = [256, 64]
    f.batch, f.heads, f.total_q, f.max_seqlen_q, f.max_pages = 3, 4, 5, 2, 8
    f.window_left, f.window_right, f.prefix_len, f.scale = -1, 0, 0, 0.125
    p.cu_groups, p.shared_lens, p.num_groups = 7 * A, 8 * A, 2
    for key, val in kw.items():
        target = p if hasattr(p, key) else f if hasattr(f, key) else c
        setattr(target, key, val)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(num_groups=0), INVALID), (dict(num_groups=4), INVALID), (dict(cu_groups=0), INVALID), (dict(shared_lens=0), INVALID),
    (dict(cu_groups=7 * A + 2), MISALIGNED), (dict(shared_lens=8 * A + 1), MISALIGNED),
    (dict(window_left=0), UNSUPPORTED), (dict(window_left=100), UNSUPPORTED), (dict(prefix_len=4), UNSUPPORTED),
    (dict(window_left=-2), INVALID), (dict(window_right=-2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(batch=0), INVALID), (dict(q=0), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(page_size=12), UNSUPPORTED),
    (dict(heads=5), INVALID), (dict(o=7 * A), INVALID), (dict(lse=8 * A), INVALID), (dict(o=A), INVALID),
    (dict(ws=7 * A), INVALID), (dict(ws=0), INVALID), (dict(ws=20 * A + 16), MISALIGNED), (dict(short=256), INVALID),
])
def test_refusals(lib, kw, code):
    ws, short = kw.pop("ws", 20 * A), kw.pop("short", 0)
    need = lib.fa2_paged_fwd_shared_workspace_bytes(ctypes.byref(_params()))
    assert lib.fa2_paged_fwd_shared(ctypes.byref(_params(**kw)), ws, need - short, None) == code
    assert lib.fa2_paged_fwd_shared(None, ws, need, None) == INVALID


def test_workspace_follows_shapes(lib):
    size = lambda **kw: lib.fa2_paged_fwd_shared_workspace_bytes(ctypes.byref(_params(**kw)))
    up = lambda x: -(-x // 256) * 256

    def expect(batch, groups, total, max_q, heads_kv, group, d):
        t, ctas, n = 128 // group, 152 if d == 256 else 304, 0
        for seqs, most in ((batch, min(max_q, total)), (groups, total)):
            places = (total // t + seqs) * heads_kv
            rows = (2 * ctas + places) * group * min(t, most)
            n += up(rows * d * 4) + up(rows * 8) + up(places * 16)
        return n

    assert size() == expect(3, 2, 5, 2, 2, 2, 64)
    assert size(head_dim=256) == expect(3, 2, 5, 2, 2, 2, 256)
    assert size(batch=64, num_groups=3, total_q=64, max_seqlen_q=1) == expect(64, 3, 64, 1, 2, 2, 64)
    assert size(num_groups=0) == 0 and size(heads=5) == 0 and size(batch=2, num_groups=3) == 0
    assert size(total_q=1 << 30, max_seqlen_q=1, batch=1 << 30, num_groups=1) == 0   # more pairs than 2^31
    assert lib.fa2_paged_fwd_shared_workspace_bytes(None) == 0
    assert lib.fa2_paged_shared_params_size() == ctypes.sizeof(fa2.Fa2PagedSharedParams)


def test_binding_refuses_host_tensors(lib):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    cache = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    q = torch.zeros((5, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        fa2.fa2_paged_fwd_shared(q, cache, cache.clone(), i32(3, 8), i32(4), i32(3), i32(3), i32(2))
    with pytest.raises(TypeError):
        fa2.fa2_paged_fwd_shared(q, cache, cache.clone(), i32(3, 8), i32(4), i32(3), None, i32(2))
