"""One attention workspace, zero-filled once, for calls of any numbers of tokens and sequences: a server's batch grows and shrinks."""
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests._gpu import DEV
from tests.test_gpu_paged_attention import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 32, 128), (32, 8, 128), (32, 8, 64), (8, 1, 128)])
def test_one_workspace_for_batches_that_grow_and_shrink(Hq, Hkv, D, dtype):
    def decode(S):  # lengths that split over CTAs, another set each time
        return " ".join(f"1+{300 + (s * 977 + S * 131) % 1700}" for s in range(S))

    steps = [decode(2), decode(24), decode(1), "300+40 1+500", decode(60), decode(4), "1+900 17+300 1+20", decode(24), decode(2), "130+700", decode(60)]
    calls = [Call(seqs, Hq, Hkv, D, 32, dtype, seed=i) for i, seqs in enumerate(steps)]
    ws = torch.zeros(max(c.ws.numel() for c in calls), dtype=torch.uint8, device=DEV)
    for c in calls:
        c.ws = ws
        c.check(c.run())
    assert nt.nt_workspace_status(ws) == nt.NT_OK


@pytest.mark.parametrize("D", [64, 128])
def test_a_large_batch_behind_small_ones(D):
    """Steps of 2, 24, 1, 256, 8 and 128 sequences."""
    calls = [Call(" ".join(f"1+{200 + (s * 389 + S) % 600}" for s in range(S)), 32, 8, D, 16, "f32", seed=S) for S in (2, 24, 1, 256, 8, 128)]
    ws = torch.zeros(max(c.ws.numel() for c in calls), dtype=torch.uint8, device=DEV)
    for c in calls + calls[::-1]:
        c.ws = ws
        c.check(c.run())
