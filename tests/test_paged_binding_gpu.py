"""The paged calls as torch functions: exceptions keep torch's types, and tensors
written in place count it."""
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


def test_out_of_memory_is_torchs():
    """An output of a terabyte; the next call works."""
    p = Problem([1], [20], 4, 2, 64, "fp16", 16, seed=1)
    with pytest.raises(torch.OutOfMemoryError):
        fa2.fa2_paged_fwd(p.q.expand(2 ** 31 - 1, -1, -1), p.k, p.v, p.table, p.cu, p.lens, window_right=0)
    o, lse = p.run(window_right=0)
    assert status() == fa2.FA2_OK
    p.check(o, lse, window_right=0)


def test_writes_in_place_are_counted():
    p = Problem([2], [20], 4, 2, 64, "fp16", 16, seed=2)
    count = lambda *x: [t._version for t in x]
    o, lse = torch.empty_like(p.q), torch.empty((4, 2), device="cuda")
    read = (p.q, p.k, p.v, p.table, p.cu, p.lens)
    ws = torch.empty(fa2.fa2_paged_fwd_workspace_bytes(*read), dtype=torch.uint8, device="cuda")
    before, before_in = count(o, lse, ws), count(*read)
    p.run(o=o, lse=lse, workspace=ws, window_right=0)
    assert count(o, lse, ws) == [x + 1 for x in before] and count(*read) == before_in

    rows, slots = torch.ones((2, 2, 64), dtype=torch.float16, device="cuda"), i32([0, 1])
    before, before_in = count(p.k, p.v), count(rows, slots)
    fa2.fa2_paged_append(rows, rows, slots, p.k, p.v)
    assert count(p.k, p.v) == [x + 1 for x in before] and count(rows, slots) == before_in

    outs = dict(cu_seqlens_q=i32([0, 0]), seqlens_k=i32([0]), slots=i32([0] * 3), free_left=i32([0]))
    args = (i32([20]), i32([3]), p.table, i32([2]), i32([1]))
    before, before_in = count(p.table, *outs.values()), count(*args[:2], *args[3:])
    fa2.fa2_paged_plan(*args, p.k.shape[0], 16, 3, **outs)
    assert count(p.table, *outs.values()) == [x + 1 for x in before] and count(*args[:2], *args[3:]) == before_in
    assert status() == fa2.FA2_OK


def test_append_to_a_cache_kept_for_backward_is_noticed():
    k = torch.zeros((2, 1, 8, 64), dtype=torch.float16, device="cuda")
    v, w = torch.zeros_like(k), torch.ones_like(k, requires_grad=True)
    loss = (w * k).sum()
    row = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda")
    fa2.fa2_paged_append(row, row, i32([3]), k, v)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors_are_taken():
    with torch.inference_mode():
        p = Problem([2], [20], 4, 2, 64, "fp16", 16, seed=3)
        rows = torch.ones((2, 2, 64), dtype=torch.float16, device="cuda")
    o = torch.empty_like(p.q)
    fa2.fa2_paged_append(rows, rows, i32([0, 1]), p.k, p.v)
    p.run(o=o, window_right=0)
    fa2.fa2_paged_plan(i32([20]), i32([3]), p.table, i32([2]), i32([1]), p.k.shape[0], 16, 3)
    assert status() == fa2.FA2_OK
    p.check(o, p.run(window_right=0)[1], window_right=0)
