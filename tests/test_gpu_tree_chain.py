"""The tree-verify calls one behind the other, as a program makes them, against 64-bit references."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from synth import workloads as wl
from tests import _tree
from tests._gpu import DEV, dev, host, tiled
from tests.test_gpu_tree import attn_bound, f64, within

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


@pytest.mark.parametrize("prefix", [3, 40])
@pytest.mark.parametrize("graph", [False, True])
def test_a_whole_pass_over_a_short_sequence(prefix, graph):
    """Layout, append, attention, adjustments, acceptance, commit and counts one behind the other. The sequence is short, so the tree's rows
    weigh; the attention's reference is formed from what the append has written, which is checked against the exact
    rotation by itself, so the attention has its own bound. An attention over stale rows, or without the tree's, is far outside."""
    rs = np.random.RandomState(prefix)
    B, Hq, Hkv, D, V = 21, 8, 2, 128, 3001
    parents = _tree.parents(rs, B)
    sees = _tree.ancestors(parents)
    q, k, v = (torch.randn(B, h, D, device=DEV) for h in (Hq, Hkv, Hkv))
    k_cache, v_cache = (torch.randn(Hkv, prefix + B, D, device=DEV).bfloat16() for _ in range(2))
    k_before, v_before = k_cache.clone(), v_cache.clone()
    parent, token = dev(parents), dev(rs.permutation(V)[:B].astype(np.int32))
    ints = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    mask, pos, choice, emit, path, n, counts = ints(B, 1), ints(B), ints(B), ints(B), ints(B), ints(1), ints(V)
    f = torch.zeros(D // 2, dtype=torch.float64, device=DEV)
    q_out, out = torch.zeros(B, Hq, D, device=DEV), torch.zeros(B, Hq, D, device=DEV)
    logits = torch.randn(B, V, device=DEV)
    for node in np.flatnonzero(sees[B - 1])[1:]:  # the last node's path agrees
        logits[parents[node], int(token[node])] = 50.0
    adjusted = torch.zeros(B, V, device=DEV)
    ws_a = torch.zeros(nt.nt_tree_attention_workspace_size(B, Hq, Hkv, D, prefix), dtype=torch.uint8, device=DEV)
    ws_l = torch.zeros(nt.nt_logits_adjust_workspace_size(V, B), dtype=torch.uint8, device=DEV)
    # the commit works on copies, so that what the attention read can be looked at
    k_moved, v_moved = torch.zeros_like(k_cache), torch.zeros_like(v_cache)
    k_ptr, v_ptr = nt.pointer_array([k_moved]), nt.pointer_array([v_moved])

    def step():
        nt.nt_rope_frequencies(D, 1e4, f)
        nt.nt_tree_layout(parent, mask, pos, prefix)
        nt.nt_qk_norm_rope_append(q, k, v, None, None, 1e-6, f, 0, 1.0, q_out, k_cache, v_cache, pos=pos, row0=prefix)
        nt.nt_tree_attention(q_out, k_cache, v_cache, prefix, prefix, mask, out, ws_a)
        nt.nt_logits_adjust(logits, counts=counts, tree_mask=mask, tokens=token, repetition=1.5, out=adjusted, argmax=choice, ws=ws_l)
        nt.nt_tree_accept(parent, token, choice, emit, path, n)
        k_moved.copy_(k_cache)
        v_moved.copy_(v_cache)
        nt.nt_tree_commit(k_ptr, v_ptr, Hkv, D, prefix + B, path, n, prefix, prefix)
        nt.nt_token_counts(token, counts, index=path, n=n)

    if graph:
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    else:
        run = step
    for turn in range(2):  # the second pass finds the first one's counts
        before = host(counts).copy()
        k_cache.copy_(k_before)
        v_cache.copy_(v_before)
        out.fill_(float("nan"))
        run()
        torch.cuda.synchronize()
        assert nt.nt_workspace_status(ws_a) == nt.NT_OK
        # the append against the exact rotation: 16 + sqrt(D) / 2 roundings of a row's largest value, and bf16's
        ff = 1e4 ** (-np.arange(D // 2) * 2.0 / D)
        for got, x, half in ((f64(q_out), q, 0.0), (f64(k_cache[:, prefix:]).transpose(1, 0, 2), k, 2.0 ** -8)):
            want = _tree.rotate(f64(x), None, 0, ff, 0, 1.0, prefix - 1 + sees.sum(1))
            size = np.abs(want).max(-1, keepdims=True) * 1.5
            within(got, want, (16 + D ** 0.5 / 2) * 2.0 ** -24 * size + half * np.abs(want), "append")
        assert torch.equal(v_cache[:, prefix:], v.bfloat16().transpose(0, 1))
        assert torch.equal(k_cache[:, :prefix], k_before[:, :prefix]) and torch.equal(v_cache[:, :prefix], v_before[:, :prefix])
        want = _tree.attend(f64(q_out), f64(k_cache), f64(v_cache), prefix, prefix, sees)
        tol = attn_bound(q_out, k_cache, v_cache, prefix, sees, "f32", want)
        within(f64(out), want, tol, "out")
        for other in (_tree.attend(f64(q_out), f64(k_before), f64(v_before), prefix, prefix, sees),
                      _tree.attend(f64(q_out), f64(k_cache), f64(v_cache), prefix, prefix, np.zeros_like(sees))):
            assert (np.abs(other - want) > tol).mean() > 0.9  # what this bound tells apart
        cnt = np.tile(before.astype(np.int64), (B, 1))
        tk = host(token)
        for b in range(B):
            cnt[b, tk[sees[b]]] += 1
        wl = _tree.adjust(host(logits), cnt, 1.5, 0.0, 0.0, None, None, np.float32)
        assert np.array_equal(host(adjusted), wl) and np.array_equal(host(choice), _tree.choice(wl))
        wp, we = _tree.accept(parents, tk, host(choice))
        assert len(wp) == sees[B - 1].sum() > 1
        assert int(n) == len(wp) and host(path).tolist()[:len(wp)] == wp and host(emit).tolist()[:len(wp)] == we
        for moved, cache in ((k_moved, k_cache), (v_moved, v_cache)):
            rows = cache.clone()
            rows[:, prefix:prefix + len(wp)] = cache[:, prefix + torch.tensor(wp, device=DEV)]
            assert torch.equal(moved, rows)
        after = before.copy()
        after[tk[wp]] += 1
        assert np.array_equal(host(counts), after)


@pytest.mark.parametrize("seed", [0, 1, 2, 3])
def test_drafted_trees_save_passes(seed):
    """Texts that repeat themselves: the drafts are accepted, so there are fewer passes than tokens, with the same tokens."""
    from examples import tree_verify as ex
    model = ex.Decoder(seed=seed)
    prompt = np.random.RandomState(seed).randint(0, model.V, 40).tolist()
    one, n_one = ex.generate(model, prompt, 96, tree=False)
    many, n_many = ex.generate(model, prompt, 96, tree=True)
    assert one == many and n_one == 96
    assert n_many < n_one
