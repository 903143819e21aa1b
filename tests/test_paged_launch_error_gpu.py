"""A paged call whose launch is refused reports it once, and no later call does.

In a child process: the refused launch goes to a stream whose capture has been
invalidated on the host (by a synchronisation while capturing)."""
import os
import subprocess
import sys

import pytest
import torch

from exact_tiled_attention_fa2_gb300 import build as fa2_build

pytestmark = pytest.mark.gpu

CHILD = """
import torch
import exact_tiled_attention_fa2_gb300 as fa2
dev = dict(device="cuda", dtype=torch.float16)
q = torch.randn((1, 1, 128, 64), **dev)
o, lse = torch.empty_like(q), torch.empty((1, 1, 128), device="cuda")
row, slots = torch.ones((1, 1, 64), **dev), torch.zeros(1, device="cuda", dtype=torch.int32)
k, v = torch.zeros((2, 1, 8, 64), **dev), torch.zeros((2, 1, 8, 64), **dev)
side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
fa2.fa2_fwd(q, q, q, o, lse)
fa2.fa2_paged_append(row, row, slots, k, v)
torch.cuda.synchronize()
def refused(f):
    try:
        f()
    except RuntimeError:
        return True
    return False
with torch.cuda.stream(side):
    graph.capture_begin()
    assert refused(torch.cuda.synchronize)   # not while capturing: the capture is invalid now
    assert refused(lambda: fa2.fa2_paged_append(row, row, slots, k, v))
    assert refused(graph.capture_end)
fa2.fa2_fwd(q, q, q, o, lse)
torch.cuda.synchronize()
print("later calls work")
"""


def test_a_refused_launch_is_reported_once():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa2_build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "later calls work" in out.stdout, out.stdout + out.stderr
