"""One workspace of nt_attention_decode, zero-filled once, for a sequence that grows, is cut back and is asked about several positions."""
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests import _paged
from tests._gpu import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 1), (16, 16)])
def test_calls_of_any_lengths_on_one_workspace(Hq, Hkv):
    nt.nt_device_check()
    g = torch.Generator(device=DEV)
    g.manual_seed(Hq)
    ts, D = 9000, 128
    k, v = (torch.randn(Hkv, ts, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    calls = [(1, 100), (1, 9000), (1, 300), (4, 5000), (1, 4000), (16, 9000), (2, 700), (1, 1), (64, 8000), (3, 2500), (1, 6000), (8, 64)]
    calls += [(1, T) for T in range(2000, 8000, 371)]
    ws = torch.zeros(max(nt.nt_attention_workspace_size(B, Hq, Hkv, T) for B, T in calls), dtype=torch.uint8, device=DEV)
    table = torch.arange(ts // 16 + 1, device=DEV).view(1, -1).cpu().numpy()
    for B, T in calls:
        q = torch.randn(B, Hq, D, generator=g, device=DEV)
        out = torch.full_like(q, -7.0)
        nt.nt_attention_decode(q, k, v, B, Hq, Hkv, D, T, ts, out, ws)
        want, _ = _paged.attend(q, k, v, table, [B], [T], 16)
        # within a few 1e-6 of max |v|, the header says
        assert float((out.double() - want).abs().max()) <= 3e-5 * float(v.float().abs().max()), (B, T)
