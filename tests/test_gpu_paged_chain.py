"""The paged-cache calls one behind the other, as a server makes them, against 64-bit references: fork, extend, copy, append,
attention and beam selection of many steps, eager on a stream of their own and in a replayed graph."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests import _paged, _tree
from tests._gpu import DEV, dev, host
from tests.test_gpu_paged_attention import U16, U32, ints

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("new,page", [(1, 16), (3, 32), (40, 16)])
def test_steps_of_a_server(new, page, dtype, graph):
    rs = np.random.RandomState(new)
    G, W, Hq, Hkv, D, V, n_pages, width = 3, 4, 8, 2, 64, 3001, 260, 24
    S, ts = G * W, n_pages * page
    T = S * new + 5  # padded
    f = 1e4 ** (-np.arange(D // 2) * 2.0 / D)
    z = lambda *s, t=I32: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
    tables, lengths, refs = [z(S, width), z(S, width)], [z(S), z(S)], z(n_pages)
    parent, start, rows, pos, pairs, bad = z(S), z(S + 1), z(T), z(T), z(S, 2), z(1)
    k_pool, v_pool = (torch.full((Hkv, ts, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    kp, vp = nt.pointer_array([k_pool]), nt.pointer_array([v_pool])
    q, k, v = z(T, Hq, D, t=dtype), z(T, Hkv, D, t=dtype), z(T, Hkv, D, t=dtype)
    q_out, out = torch.empty_like(q), torch.full_like(q, -7.0)
    logits, scores = z(S, V, t=torch.float32), z(S, t=torch.float32)
    token, score, done = z(S), z(S, t=torch.float32), z(S)
    inv_freq = dev(f)
    ws_a = torch.zeros(nt.nt_paged_attention_workspace_size(T, S, Hq, Hkv, D), dtype=torch.uint8, device=DEV)
    ws_b = torch.zeros(nt.nt_beam_select_workspace_size(V, S), dtype=torch.uint8, device=DEV)

    def step():
        nt.nt_page_fork(tables[0], lengths[0], parent, refs, page, tables[1], lengths[1])
        nt.nt_page_extend(tables[1], lengths[1], refs, start, page, rows, pos, pairs, n_bad=bad)
        nt.nt_page_copy(kp, vp, Hkv, D, ts, page, pairs)
        nt.nt_qk_norm_rope_append(q, k, v, None, None, 1e-6, inv_freq, nt.NT_ROPE_HALF, 1.0, q_out, k_pool, v_pool, pos=pos, rows=rows)
        nt.nt_paged_attention(q_out, k_pool, v_pool, page, tables[1], start, lengths[1], out, ws_a, max_new=new)
        nt.nt_beam_select(logits, scores, W, parent, token, score, ws_b, done_out=done, eos=7)
        tables[0].copy_(tables[1])
        lengths[0].copy_(lengths[1])
        scores.copy_(score)

    stream, g = torch.cuda.Stream(), None
    table, length, count = np.full((S, width), -1, dtype=np.int32), np.zeros(S, dtype=np.int32), np.zeros(n_pages, dtype=np.int32)
    up, total = np.full(S, -1), np.zeros(S, dtype=np.float32)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        parent.fill_(-1)
        for t in range(12):
            counts = rs.randint(0, new + 1, S) if t else np.full(S, new)
            n = int(counts.sum())
            start.copy_(ints(np.concatenate(([0], np.cumsum(counts)))))
            for x in (q, k, v):
                x.copy_(torch.randn(x.shape, device=DEV))
            logits.copy_(torch.randn(S, V, device=DEV) * 2)
            out.fill_(-7.0)
            if graph and t == 2:
                stream.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    step()
            g.replay() if g else step()
            stream.synchronize()
            # the tables
            table, length, count = _paged.fork(table, length, up, count, page)
            table, length, count, r, p, copies, _ = _paged.extend(table, length, count, counts.tolist(), page)
            assert np.array_equal(host(tables[1]), table) and np.array_equal(host(lengths[1]), length) and np.array_equal(host(refs), count)
            assert np.array_equal(host(rows)[:n], r) and (host(rows)[n:] == -1).all() and np.array_equal(host(pairs), copies)
            # what was appended, and the rows that the queries see
            want_k = _tree.rotate(k[:n].double().cpu().numpy(), None, 0.0, f, 0, 1.0, p)
            got_k = k_pool[:, torch.from_numpy(r.astype(np.int64)).to(DEV)].double().cpu().numpy().transpose(1, 0, 2)
            assert (np.abs(got_k - want_k) <= U16 * np.abs(want_k) + 32 * U32 * np.abs(want_k).max(initial=0.0)).all()
            want, size = _paged.attend(q_out[:n], k_pool, v_pool, table, counts.tolist(), length, page)
            norm = float(q_out[:n].double().norm(dim=-1).max() * 16.0) / D ** 0.5 if n else 0.0  # keys of 64 dimensions: |k| below 16
            tol = (4 * U32 * (D ** 0.5 * norm + 16) + (2.0 ** -15 if dtype == torch.float32 else 2 * U16 + 2.0 ** -12)) * size
            tol = tol + (2 * U32 if dtype == torch.float32 else U16) * want.abs()
            assert ((out[:n].double() - want).abs() <= tol).all() and (out[n:] == -7.0).all()
            # the beams
            want = _paged.beam(host(logits), total, W, W, eos=7)
            assert np.array_equal(host(parent), want[0]) and np.array_equal(host(token), want[1]) and np.array_equal(host(done), want[3])
            assert np.abs(host(score) - want[2]).max() <= 2.0 ** -22 * max(np.abs(want[2]).max(), float(logits.abs().max()))
            up, total = want[0], host(score).copy()
    assert nt.nt_workspace_status(ws_a) == nt.NT_OK


def test_two_streams_with_workspaces_of_their_own():
    """Attention and selection on two streams at once give what they give alone."""
    calls = []
    for seed in (0, 1):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        n = [1, 1, 60][seed:seed + 2]
        S, T = len(n), sum(n)
        length = np.array([500 + 40 * seed, 900])[:S] + np.array(n)
        held = [_paged.pages_of(x, 16) for x in length]
        table = np.full((S, max(held)), -1)
        at = 0
        for s, h in enumerate(held):
            table[s, :h] = np.arange(at, at + h)
            at += h
        q = torch.randn(T, 8, 128, generator=gen, device=DEV)
        k, v = (torch.randn(2, at * 16, 128, generator=gen, device=DEV).bfloat16() for _ in range(2))
        calls.append(dict(q=q, k_pool=k, v_pool=v, page=16, table=ints(table), q_start=ints(np.concatenate(([0], np.cumsum(n)))), length=ints(length),
                          out=torch.empty_like(q), max_new=max(n),
                          ws=torch.zeros(nt.nt_paged_attention_workspace_size(T, S, 8, 2, 128), dtype=torch.uint8, device=DEV)))
    want = []
    for c in calls:
        nt.nt_paged_attention(**c)
        torch.cuda.synchronize()
        want.append(c["out"].clone())
        c["out"].zero_()
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(50):
        for c, st in zip(calls, streams):
            nt.nt_paged_attention(**c, stream=st)
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert torch.equal(c["out"], w)


def test_attention_directly_behind_a_projection_that_holds_tensor_memory():
    """The attention's launch begins while the projection before it runs; both allocate tensor memory."""
    from synth import workloads as wl
    from tests._gpu import tiled
    B, Hq, Hkv, D, K, before = 16, 32, 8, 128, 2048, 500
    N = Hq * D
    p = wl.projection(9, 0, 0, N, K, B, seed=1)
    w, s_w = tiled(p.w_plain, N, K), dev(p.s_w)
    codes, s_x = torch.empty(B, K, dtype=torch.int8, device=DEV), torch.empty(B, device=DEV)
    nt.nt_quantize_act(dev(p.x), codes, s_x)
    k, v = (torch.randn(Hkv, 1024, D, device=DEV).bfloat16() for _ in range(2))
    ws_p = torch.zeros(nt.nt_ternary_gemm_workspace_size(N, K, B, nt.NT_LAYOUT_TILED), dtype=torch.uint8, device=DEV)
    ws_a = torch.zeros(nt.nt_paged_attention_workspace_size(B, 1, Hq, Hkv, D), dtype=torch.uint8, device=DEV)
    q, out = torch.empty(B, Hq, D, device=DEV), torch.empty(B, Hq, D, device=DEV)
    table, start, length = ints(np.arange(64)[None]), ints([0, B]), ints([before + B])

    def step(wait=lambda: None):
        nt.nt_ternary_gemm(w, nt.NT_LAYOUT_TILED, s_w, N, K, codes, s_x, B, q, ws=ws_p)
        wait()
        nt.nt_paged_attention(q, k, v, 16, table, start, length, out, ws_a, max_new=B)
        wait()

    step(torch.cuda.synchronize)
    want = out.clone()
    for _ in range(300):
        step()
    torch.cuda.synchronize()
    assert nt.nt_workspace_status(ws_p) == nt.NT_OK and nt.nt_workspace_status(ws_a) == nt.NT_OK
    assert torch.equal(out, want)
