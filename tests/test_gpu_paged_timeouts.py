"""Waits of the paged attention for few rows that run out: no copies are issued (a host-side hook), every wait ends after 20 ms and is
reported until the workspace is zero-filled again. Nothing hangs, and no GPU fault is involved."""
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests.test_gpu_paged_attention import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (8, 1, 128), (32, 8, 128)])
@pytest.mark.parametrize("seqs", ["1+0", "1+4000", "1+300 1+7 1+1000", "1+90 " * 60, "1+600 40+200 2+3"])
def test_a_wait_that_runs_out(seqs, Hq, Hkv, D, dtype):
    c = Call(seqs, Hq, Hkv, D, 16, dtype)
    try:
        nt.nt_set_test_fault(6, 20.0)
        c.run()
        torch.cuda.synchronize()
    finally:
        nt.nt_set_test_fault(0)
    assert nt.nt_workspace_status(c.ws) == nt.NT_ERR_TIMEOUT
    c.run()  # still reported; what comes out is not said
    assert nt.nt_workspace_status(c.ws) == nt.NT_ERR_TIMEOUT
    c.ws.zero_()
    c.check(c.run())
    assert nt.nt_workspace_status(c.ws) == nt.NT_OK
