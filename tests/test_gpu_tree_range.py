"""The tree-verify operators over the whole range that their calls accept: long sums, groups of rows, a whole pass in the
order in which a program makes it. References are in 64 bits; tolerances count roundings (fp32 2^-24, bf16 2^-8)."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests import _tree
from tests._gpu import DEV, dev, host
from tests.test_gpu_tree import attend_64, attn_bound, attn_inputs, run_adjust, run_attend, within
from tests.test_tree_plans_cpu import GROUPED_ROWS

pytestmark = pytest.mark.gpu
U32, U16 = 2.0 ** -24, 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- attention -------------------------------------------------------------------------------
@pytest.mark.parametrize("B,D,tiles,dtype", [(36, 128, 1600, "bf16"), (70, 128, 1001, "bf16"), (36, 64, 1600, "bf16"),
                                             (70, 64, 1601, "bf16"), (36, 64, 1600, "f32"), (70, 128, 1001, "f32")])
def test_attention_sums_of_one_sign_keep_their_bits(B, D, tiles, dtype):
    """A head to a block and values of one sign: a thousand tiles and more go to one accumulator, and what the tensor core cuts
    off its sums cannot cancel. A sum loses at most one step, 2^-23, per 16 keys and weight term while it stays in tensor
    memory: 12 per tile over 8 tiles with fp32 queries, 8 over 16 with bf16 ones. What it is added to rounds to nearest.
    A bf16 output has rounded, so the loss shows in the mean over many outputs, whose values spread over a binade (a scale to
    every head and dimension): the bf16 rounding and the weights' own (2^-18 each) have no side and are allowed five standard
    deviations of that mean."""
    Hkv, prefix = 152, 64 * (tiles - (B + 63) // 64)
    g = torch.Generator(device=DEV)
    g.manual_seed(B + D)
    ts = prefix + B
    q = torch.randn(B, Hkv, D, generator=g, device=DEV).mul_(0.5).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    k, v = (torch.empty(Hkv, ts, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for h in range(Hkv):
        k[h] = torch.randn(ts, D, generator=g, device=DEV).mul_(0.25).bfloat16()
        v[h] = ((1 + torch.rand(ts, D, generator=g, device=DEV) * 0.5) * torch.rand(D, generator=g, device=DEV).exp2()).bfloat16()
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(B), B))
    ws = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hkv, Hkv, D, prefix), dtype=torch.uint8, device=DEV)
    outs = []
    for _ in range(3):
        out = torch.empty_like(q)
        nt.nt_tree_attention(q, k, v, prefix, prefix, dev(_tree.pack(sees)), out, ws)
        torch.cuda.synchronize()
        assert nt.nt_workspace_status(ws) == nt.NT_OK
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    off = np.empty((Hkv, B, D))
    for h in range(Hkv):
        s = q[:, h].double() @ k[h].double().T / D ** 0.5
        s[:, prefix:] = s[:, prefix:].masked_fill(~dev(sees), float("-inf"))
        want = s.softmax(-1) @ v[h].double()
        off[h] = host(outs[0][:, h].double() / want - 1)
    loss = (8 * 16 if dtype == "bf16" else 12 * 8) * 2 * U32
    # scores (sqrt(D) roundings of |q| |k| / sqrt(D), twice: in a weight and in the weights' sum), sums, exponentials and quotient
    rest = 2 * U32 * (2 * 0.5 * 0.25 * D ** 0.5 * 1.5 + tiles ** 0.5 + 16)
    mean, worst = float(off.mean()), float(np.abs(off).max())
    if dtype == "f32":
        assert worst <= loss + rest, (worst, loss, rest)
    else:
        spread = off.mean(1).std() / (Hkv * D) ** 0.5  # a head's nodes have much the same sums: one sample for all of them
        assert abs(mean) <= loss + 5 * spread, (mean, loss, spread, worst)
        assert worst <= U16 + loss + rest + 2.0 ** -18, worst


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [36, 70, 133])
@pytest.mark.parametrize("kind", ["random", "rise", "fall", "steps"])
def test_attention_bf16_about_the_points_where_sums_are_taken(B, D, kind):
    """A head to a block, every tile count about the multiples of 16; the reference stays, rises with every tile, falls, or jumps at
    the tiles about those points."""
    Hkv = 160
    for tiles in (15, 16, 17, 18, 31, 32, 33, 34, 47, 48, 49, 50, 64, 65):
        prefix = max(0, 64 * tiles - 64 * ((B + 63) // 64) - (tiles % 3) * 9)
        q, k, v = attn_inputs(B, Hkv, Hkv, D, prefix, 0, "bf16", seed=tiles)
        if kind != "random":
            at = torch.arange(k.shape[1], device=DEV)
            ramp = {"rise": at / k.shape[1] * 40, "fall": 40 - at / k.shape[1] * 40, "steps": (at // 64 + 1) // 16 * 12.0}[kind]
            u = q.float().mean(0)
            k = (k * 0.1 + ramp[None, :, None] * (u / u.norm(dim=-1, keepdim=True))[:, None]).bfloat16()
        sees = _tree.ancestors(_tree.parents(np.random.RandomState(tiles), B))
        out = run_attend(q, k, v, prefix, prefix, sees, runs=2)
        want = attend_64(q, k, v, prefix, prefix, sees)
        within(f64(out), want, attn_bound(q, k, v, prefix, sees, "bf16", want), (kind, tiles))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hkv,prefix", [(70, 200, 2500), (40, 170, 3100), (255, 8, 9000)])
def test_attention_bf16_sums_in_shares(B, Hkv, prefix, D):
    """Blocks that begin and end within a tile of rows, each piece with sums of its own; a node's infinity reaches it alone."""
    q, k, v = attn_inputs(B, Hkv * (1 if Hkv > 8 else 4), Hkv, D, prefix, 1, "bf16", seed=B)
    ramp = torch.linspace(0, 30, k.shape[1], device=DEV)
    u = q.float().view(B, Hkv, -1, D).mean((0, 2))
    k = (k * 0.1 + ramp[None, :, None] * (u / u.norm(dim=-1, keepdim=True))[:, None]).bfloat16()
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(B), B))
    sees[:, B - 1] = False
    sees[B - 1, B - 1] = True
    v[:, prefix + B] = float("inf")
    out = f64(run_attend(q, k, v, prefix, prefix + 1, sees, runs=2))
    want = attend_64(q, k, v.nan_to_num(0, 0, 0), prefix, prefix + 1, sees)
    assert np.isposinf(out[B - 1]).all()
    within(out[:-1], want[:-1], attn_bound(q, k, v, prefix, sees, "bf16", want)[:-1])


def test_attention_bf16_timeout_is_reported_with_sums_aside():
    q, k, v = attn_inputs(70, 160, 160, 128, 3000, 0, "bf16")
    sees = _tree.ancestors(_tree.parents(np.random.RandomState(6), 70))
    want = run_attend(q, k, v, 3000, 3000, sees)
    ws = torch.zeros(nt.nt_tree_attention_workspace_size(70, 160, 160, 128, 3000), dtype=torch.uint8, device=DEV)
    mask, out = dev(_tree.pack(sees)), torch.empty_like(q)
    try:
        nt.nt_set_test_fault(5, 20.0)
        nt.nt_tree_attention(q, k, v, 3000, 3000, mask, out, ws)
        torch.cuda.synchronize()
    finally:
        nt.nt_set_test_fault(0)
    assert nt.nt_workspace_status(ws) == nt.NT_ERR_TIMEOUT
    ws.zero_()
    nt.nt_tree_attention(q, k, v, 3000, 3000, mask, out, ws)
    torch.cuda.synchronize()
    assert nt.nt_workspace_status(ws) == nt.NT_OK and torch.equal(out, want)


# ---- logits ----------------------------------------------------------------------------------
@pytest.mark.parametrize("rep", [2e-9, 5.9e-8, 2.0 ** -24, 6.1e-8, 1.6e7, 2.0 ** 24, 1.7e7, 9e8, 1.5e-9, 9.99e8])
def test_adjust_quotients_where_they_leave_the_range(rep):
    """Values whose quotients overflow, are subnormal or lie next to either, one by one (listed tokens) and all together."""
    rs = np.random.RandomState(3)
    sig = np.concatenate([1 + rs.rand(4000), [1.0, 2 - 2.0 ** -23, 1.5, 1.4142135]]).astype(np.float32)
    x = np.concatenate([np.ldexp(sig, e) for e in (-149, -126, -125, -101, -100, -99, 0, 98, 99, 100, 126, 127)]).astype(np.float32)
    x = np.concatenate([x, -x, np.float32([0.0, -0.0, np.inf, -np.inf])])
    with np.errstate(over="ignore", under="ignore"):
        r = np.float32(rep)
        want = np.where(x > 0, x / r, x * r)
    for every in (1, 37):
        counts = (np.arange(x.size) % every == 0).astype(np.int32)
        out, arg = torch.empty(1, x.size, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
        ws = torch.zeros(nt.nt_logits_adjust_workspace_size(x.size, 1), dtype=torch.uint8, device=DEV)
        nt.nt_logits_adjust(dev(x[None]), counts=dev(counts), repetition=rep, out=out, argmax=arg, ws=ws)
        full = np.where(counts > 0, want, x)[None]
        assert np.array_equal(host(out), full)
        assert np.array_equal(host(arg), _tree.choice(full))


@pytest.mark.parametrize("group,B,V", GROUPED_ROWS)
@pytest.mark.parametrize("kind", ["paths", "rows", "in place"])
def test_adjust_rows_in_groups(group, B, V, kind):
    """Several rows to a block: the ring of rows goes round, every row has its own path, allowed words and (rows) counts and
    biases, the last group is ragged; against the fp32 evaluation step by step, twice on one workspace."""
    assert group > 1 and torch.cuda.get_device_properties(DEV).multi_processor_count == 152
    run_adjust(B, V, True, "row", True, seed=B, strided=kind == "rows", inplace=kind == "in place", want_out=V != 40004)


@pytest.mark.parametrize("V", [151936, 151935])
def test_adjust_groups_with_the_same_tokens_on_many_nodes(V):
    """A token on several nodes of a path counts once for each, in every row of a group, listed (few used tokens) or not."""
    rs = np.random.RandomState(V)
    B = 64
    x = (rs.randn(B, V) * 4).astype(np.float32)
    sees = _tree.ancestors(_tree.parents(rs, B))
    for every in (3000, 3):
        counts = np.where(np.arange(V) % every == 0, 1 + rs.randint(0, 3, V), 0).astype(np.int32)
        tokens = rs.choice([7, 8, 2000, 2047, 2048, V - 1, V // 2], B).astype(np.int32)
        full = np.stack([counts + np.bincount(tokens[s], minlength=V) for s in sees]).astype(np.int32)
        want = _tree.adjust(x, full, 1.3, 0.25, -0.5, None, None, np.float32)
        out, arg = torch.empty(B, V, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
        ws = torch.zeros(nt.nt_logits_adjust_workspace_size(V, B), dtype=torch.uint8, device=DEV)
        for _ in range(2):
            nt.nt_logits_adjust(dev(x), counts=dev(counts), tree_mask=dev(_tree.pack(sees)), tokens=dev(tokens), repetition=1.3,
                                frequency=0.25, presence=-0.5, out=out, argmax=arg, ws=ws)
            assert np.array_equal(host(out), want) and np.array_equal(host(arg), _tree.choice(want))
            assert not ws.any()
