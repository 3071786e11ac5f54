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


def test_one_tensor_of_the_host_among_those_of_the_gpu_is_refused():
    """On the host, before anything is launched: the address would go to the kernel."""
    i32 = torch.int32
    q, c = torch.zeros(2, 4, 64, device=DEV), torch.zeros(2, 16, 64, dtype=torch.bfloat16, device=DEV)
    mask, b, ws = (torch.zeros(*s, dtype=t, device=DEV) for s, t in (((2, 1), i32), ((2,), i32), ((4096,), torch.uint8)))
    for bad in (dict(mask=mask.cpu()), dict(q=q.cpu()), dict(k_cache=c.cpu()), dict(v_cache=c.cpu()), dict(out=q.cpu()), dict(ws=ws.cpu())):
        args = dict(q=q, k_cache=c, v_cache=c, prefix=4, tree_row0=4, mask=mask, out=q, ws=ws)
        with pytest.raises(nt.NtError, match=f"{'|'.join(bad)} must be a CUDA tensor"):
            nt.nt_tree_attention(**{**args, **bad})
    for bad in ("counts", "bias", "allowed", "out", "argmax", "ws"):
        args = dict(counts=torch.zeros(9, dtype=i32, device=DEV), bias=torch.zeros(9, device=DEV), allowed=torch.zeros(1, dtype=i32, device=DEV),
                    out=torch.zeros(2, 9, device=DEV), argmax=b, ws=ws)
        args[bad] = args[bad].cpu()
        with pytest.raises(nt.NtError, match=f"{bad} must be a CUDA tensor"):
            nt.nt_logits_adjust(torch.zeros(2, 9, device=DEV), **args)
    with pytest.raises(nt.NtError, match="n must be a CUDA tensor"):
        nt.nt_token_counts(b, torch.zeros(9, dtype=i32, device=DEV), n=torch.ones(1, dtype=i32))
    with pytest.raises(nt.NtError, match="the caches must be a CUDA tensor"):
        nt.nt_tree_commit(nt.pointer_array([c.cpu()]), nt.pointer_array([c.cpu()]), 2, 64, 16, b, b[:1], 4, 4)
    with pytest.raises(OverflowError):
        nt.nt_tree_accept(b, b, b, b, b, b[:1], stream=1 << 80)
