"""The attention kernels' bounded wait (a limit in cycles of the SM's clock, 2e9): a barrier
that nothing completes ends in an error word and a raised abort flag, other waits see the flag,
and the context stays usable."""
import ctypes
import os
import subprocess

import pytest
import torch

import __graft_entry__ as g
from block_draft_proposal_gb300 import dflash2
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def probe(cuda, tmp_path_factory):
    so = str(tmp_path_factory.mktemp("probe") / "attention_wait_probe.so")
    cmd = [g._nvcc(), *g.NVCC_FLAGS, "-shared", os.path.join(HERE, "attention_wait_probe.cu"), "-o", so]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(so)
    lib.attention_wait_probe.argtypes = [ctypes.c_void_p] * 3
    lib.attention_wait_probe.restype = ctypes.c_int
    return lib


def test_a_wait_that_nothing_ends_gives_up(cuda, probe):
    err = torch.zeros(1, dtype=torch.int32, device=cuda)
    elapsed = torch.zeros(2, dtype=torch.int64, device=cuda)
    result = torch.full((5,), -1, dtype=torch.int32, device=cuda)
    torch.cuda.synchronize()
    assert probe.attention_wait_probe(err.data_ptr(), elapsed.data_ptr(), result.data_ptr()) == 0
    assert result.tolist() == [1, 0, 1, 0, 1]
    assert int(err.item()) == dflash2.DEVERR_TIMEOUT
    first, second = (x / 1e9 for x in elapsed.tolist())
    assert 0.9 <= first < 5.0 and second < 0.1, (first, second)
    c = Case([3], [50], 4, 2, 64, 16, seed=1)
    out, lse, err = c.run()
    assert int(err.item()) == 0
    c.check(out, lse)
