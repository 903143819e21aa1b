"""The paged calls as torch functions: exceptions keep torch's types."""
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
