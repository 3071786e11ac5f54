"""The tree-verify calls one behind the other, as a program makes them, against 64-bit references."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from synth import workloads as wl
from tests import _tree
from tests._gpu import DEV, dev, tiled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [4, 16])
def test_attention_directly_behind_a_projection(B):
    """The tensor-core projection and the attention both hold tensor memory, and the attention's launch begins while the
    projection runs: queries straight from the projection, many times over, give what they give one call at a time."""
    Hq, Hkv, D, K, prefix = 32, 8, 128, 2048, 500
    N = Hq * D
    p = wl.projection(9, 0, 0, N, K, B, seed=1)
    w, s_w = tiled(p.w_plain, N, K), dev(p.s_w)
    codes, s_x = torch.empty(B, K, dtype=torch.int8, device=DEV), torch.empty(B, device=DEV)
    nt.nt_quantize_act(dev(p.x), codes, s_x)
    k, v = (torch.randn(Hkv, prefix + B, D, device=DEV).bfloat16() for _ in range(2))
    mask = dev(_tree.pack(np.tril(np.ones((B, B), bool))))
    ws_p = torch.zeros(nt.nt_ternary_gemm_workspace_size(N, K, B, nt.NT_LAYOUT_TILED), dtype=torch.uint8, device=DEV)
    ws_a = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hq, Hkv, D, prefix), dtype=torch.uint8, device=DEV)
    q, out = torch.empty(B, Hq, D, device=DEV), torch.empty(B, Hq, D, device=DEV)

    def step(wait=lambda: None):
        nt.nt_ternary_gemm(w, nt.NT_LAYOUT_TILED, s_w, N, K, codes, s_x, B, q, ws=ws_p)
        wait()
        nt.nt_tree_attention(q, k, v, prefix, prefix, mask, out, ws_a)
        wait()

    step(torch.cuda.synchronize)
    want = out.clone()
    for _ in range(300):
        step()
    torch.cuda.synchronize()
    assert nt.nt_workspace_status(ws_p) == nt.NT_OK and nt.nt_workspace_status(ws_a) == nt.NT_OK
    assert torch.equal(out, want)
