"""Refusals of the paged-cache calls: every malformed argument is answered on the host before any launch (no GPU needed), with
the status the header states; well-formed ones get as far as the device check. And what the binding refuses."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import build as nt_build
from packed_weight_gemv_gb300 import nt
from tests import _paged
from tests.test_tree_cpu import ALIGN, INV, P, UNSUP, WS, call, reaches_device

I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    nt_build.build()
    return nt.load_library()


FORK = dict(table=P[0], length=P[1], S=4, W=8, parent=P[2], So=4, page=16, refs=P[3], n=50, to=P[4], lo=P[5], bad=P[6], stream=None)
EXTEND = dict(table=P[0], length=P[1], S=4, W=8, start=P[2], T=9, page=16, refs=P[3], n=50, rows=P[4], pos=P[5], pairs=P[6], bad=None, stream=None)
COMPACT = dict(refs=P[0], n=50, table=P[1], length=P[2], S=4, W=8, page=16, pairs=P[3], m=25, used=P[4], bad=None, ws=P[5], bytes=1 << 20, stream=None)
PAGED = dict(q=P[0], dtype=0, qs=1024, k=P[1], v=P[2], T=5, S=2, Hq=8, Hkv=2, D=128, page=16, ts=256, table=P[3], W=8, start=P[4], length=P[5],
             most=0, window=0, cap=0.0, slopes=None, out=P[6], bad=None, ws=P[7], bytes=1 << 40, stream=None)
BEAM = dict(x=P[0], s=P[1], N=8, W=4, V=100, K=4, done=P[2], eos=5, lens=P[3], alpha=0.6, parent=P[4], token=P[5], score=P[6], dout=P[7],
            ws=P[8], bytes=1 << 30, stream=None)


def copy_args(**bad):
    import ctypes
    k, v = ((ctypes.c_void_p * 2)(*bad.pop(n, (P[a], P[a + 1]))) for n, a in (("k", 0), ("v", 2)))
    return dict(dict(k=k, v=v, L=2, Hkv=2, D=64, ts=100, page=16, pairs=P[4], n=3, stream=None), **bad)


@pytest.mark.parametrize("bad,status", [
    (dict(table=None), INV), (dict(length=None), INV), (dict(parent=None), INV), (dict(refs=None), INV), (dict(to=None), INV), (dict(lo=None), INV),
    (dict(S=0), INV), (dict(S=4097), INV), (dict(So=0), INV), (dict(So=4097), INV), (dict(W=0), INV), (dict(n=0), INV), (dict(page=8), INV),
    (dict(page=48), INV), (dict(page=512), INV), (dict(page=256, n=1 << 23), INV), (dict(table=P[0] + 2), ALIGN), (dict(refs=P[3] + 1), ALIGN),
    (dict(bad=P[6] + 2), ALIGN), (dict(to=P[0]), INV), (dict(to=P[0] + 4 * 31), INV), (dict(to=P[0] - 4), INV), (dict(lo=P[1]), INV), (dict(lo=P[2]), INV),
    (dict(to=P[2] - 8), INV)])
def test_fork_refusals(lib, bad, status):
    assert call(lib.nt_page_fork, FORK, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(table=None), INV), (dict(length=None), INV), (dict(start=None), INV), (dict(refs=None), INV), (dict(rows=None), INV), (dict(pos=None), INV),
    (dict(pairs=None), INV), (dict(S=0), INV), (dict(S=4097), INV), (dict(T=0), INV), (dict(T=(1 << 20) + 1), INV), (dict(W=0), INV), (dict(n=0), INV),
    (dict(page=0), INV), (dict(page=24), INV), (dict(pos=P[5] + 1), ALIGN), (dict(pairs=P[6] + 2), ALIGN), (dict(bad=P[7] + 2), ALIGN)])
def test_extend_refusals(lib, bad, status):
    assert call(lib.nt_page_extend, EXTEND, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(k=(None, P[1])), INV), (dict(v=(P[2], None)), INV), (dict(k=(P[0] + 8, P[1])), ALIGN), (dict(pairs=None), INV), (dict(pairs=P[4] + 1), ALIGN),
    (dict(L=0), INV), (dict(Hkv=0), INV), (dict(Hkv=65536), INV), (dict(D=12), UNSUP), (dict(D=264), UNSUP), (dict(ts=15), INV), (dict(page=17), INV),
    (dict(n=0), INV)])
def test_copy_refusals(lib, bad, status):
    assert call(lib.nt_page_copy, copy_args(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(refs=None), INV), (dict(table=None), INV), (dict(length=None), INV), (dict(pairs=None), INV), (dict(used=None), INV), (dict(S=0), INV),
    (dict(n=0), INV), (dict(m=24), INV), (dict(page=100), INV), (dict(W=0), INV), (dict(used=P[4] + 2), ALIGN), (dict(ws=None), WS), (dict(ws=P[5] + 4), WS),
    (dict(bytes=455), WS)])
def test_compact_refusals(lib, bad, status):
    assert call(lib.nt_page_compact, COMPACT, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(table=None), INV), (dict(start=None), INV), (dict(length=None), INV),
    (dict(out=None), INV), (dict(dtype=2), INV), (dict(D=96), UNSUP), (dict(T=0), INV), (dict(T=(1 << 20) + 1), INV), (dict(S=0), INV), (dict(S=4097), INV),
    (dict(Hkv=0), INV), (dict(Hq=9), INV), (dict(Hq=130, Hkv=2), INV), (dict(T=1 << 20, Hq=32, qs=4096), INV), (dict(page=20), INV), (dict(ts=15), INV),
    (dict(W=0), INV), (dict(most=-1), INV), (dict(window=-1), INV), (dict(cap=-1.0), INV), (dict(cap=float("inf")), INV), (dict(cap=float("nan")), INV),
    (dict(cap=2.0 ** -101), INV), (dict(cap=2.0 ** 101), INV),
    (dict(qs=1028), ALIGN), (dict(qs=1016), INV), (dict(out=P[0], qs=2048), INV), (dict(q=P[0] + 8), ALIGN), (dict(k=P[1] + 2), ALIGN),
    (dict(v=P[2] + 8), ALIGN), (dict(out=P[6] + 4), ALIGN), (dict(table=P[3] + 1), ALIGN), (dict(slopes=P[8] + 2), ALIGN), (dict(bad=P[8] + 2), ALIGN),
    (dict(ws=None), WS), (dict(ws=P[7] + 8), WS), (dict(bytes=100), WS)])
def test_attention_refusals(lib, bad, status):
    assert call(lib.nt_paged_attention, PAGED, **bad) == status


def test_attention_workspace_is_what_the_call_wants(lib):
    for T, S, Hq, Hkv, D in ((1, 1, 1, 1, 64), (1, 1, 32, 8, 128), (8191, 5, 32, 8, 128), (64, 64, 40, 8, 128), (300, 4096, 8, 1, 64)):
        n = nt.nt_paged_attention_workspace_size(T, S, Hq, Hkv, D)
        a = dict(T=T, S=S, Hq=Hq, Hkv=Hkv, D=D, qs=Hq * D)
        assert call(lib.nt_paged_attention, PAGED, **a, bytes=n - 1) == WS
        if not torch.cuda.is_available():
            assert reaches_device(call(lib.nt_paged_attention, PAGED, **a, bytes=n))
    for bad in ((0, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 1, 9, 2, 128), (1, 1, 8, 0, 128), (1, 1, 8, 2, 32), (1, 1, 130, 2, 128)):
        with pytest.raises(nt.NtError):
            nt.nt_paged_attention_workspace_size(*bad)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), INV), (dict(s=None), INV), (dict(parent=None), INV), (dict(token=None), INV), (dict(score=None), INV), (dict(N=0), INV),
    (dict(N=9), INV), (dict(N=65540), INV), (dict(W=0), INV), (dict(W=65, N=65), INV), (dict(V=0), INV), (dict(V=(1 << 24) + 1), INV), (dict(K=0), INV),
    (dict(K=65), INV), (dict(eos=100), INV), (dict(eos=-2), INV), (dict(eos=-1), INV), (dict(alpha=-0.1), INV), (dict(alpha=17.0), INV), (dict(alpha=4.01), INV),
    (dict(score=P[1]), INV), (dict(dout=P[2]), INV), (dict(parent=P[3]), INV), (dict(token=P[0] + 64), INV),
    (dict(alpha=float("nan")), INV), (dict(lens=None), INV), (dict(x=P[0] + 2), ALIGN), (dict(done=P[2] + 1), ALIGN), (dict(dout=P[7] + 2), ALIGN),
    (dict(ws=None), WS), (dict(ws=P[8] + 8), WS), (dict(bytes=300), WS)])
def test_beam_refusals(lib, bad, status):
    assert call(lib.nt_beam_select, BEAM, **bad) == status


def test_well_formed_arguments_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real: only where there is no device")
    for fn, good in ((lib.nt_page_fork, FORK), (lib.nt_page_extend, EXTEND), (lib.nt_page_copy, copy_args()), (lib.nt_page_compact, COMPACT),
                     (lib.nt_paged_attention, PAGED), (lib.nt_beam_select, BEAM)):
        assert reaches_device(call(fn, good))
    for ok in (dict(done=None, eos=-1), dict(alpha=0.0, lens=None), dict(dout=None), dict(K=64, W=8)):
        assert reaches_device(call(lib.nt_beam_select, BEAM, **ok))
    for ok in (dict(T=1, qs=0), dict(out=P[0]), dict(slopes=P[9], cap=30.0, window=7), dict(most=1 << 30), dict(dtype=1, qs=4096)):
        assert reaches_device(call(lib.nt_paged_attention, PAGED, **ok))


def test_the_binding_refuses_shapes_types_and_places():
    z = lambda *s, t=I32: torch.zeros(*s, dtype=t)  # noqa: E731
    f32, bf = torch.float32, torch.bfloat16
    table, n, refs, start = z(3, 4), z(3), z(9), z(4)
    ws = z(1 << 22, t=torch.uint8)
    q, k = z(5, 4, 64, t=f32), z(2, 64, 64, t=bf)
    caches = nt.pointer_array([k, k])
    calls = [
        (nt.nt_page_fork, dict(table=table, length=n, parent=n.clone(), refs=refs, page=16, table_out=table.clone(), length_out=n.clone())),
        (nt.nt_page_extend, dict(table=table, length=n, refs=refs, q_start=start, page=16, rows=z(5), pos=z(5), pairs=z(3, 2))),
        (nt.nt_page_compact, dict(refs=refs, table=table, length=n, page=16, pairs=z(5, 2), n_used=z(1), ws=ws)),
        (nt.nt_paged_attention, dict(q=q, k_pool=k, v_pool=k, page=16, table=table, q_start=start, length=n, out=q.clone(), ws=ws, slopes=z(4, t=f32))),
        (nt.nt_beam_select, dict(logits=z(6, 50, t=f32), scores=z(6, t=f32), beams=3, parent=z(8), token=z(8), score=z(8, t=f32), ws=ws, done=z(6),
                                 done_out=z(8), eos=3, lengths=z(6), alpha=1.0)),
        (nt.nt_page_copy, dict(k_caches=caches, v_caches=caches, Hkv=2, D=64, t_stride=64, page=16, pairs=z(3, 2))),
    ]
    for fn, args in calls:
        with pytest.raises(nt.NtError, match="must be a CUDA tensor"):  # all else is in order
            fn(**args, stream=0)
        for name, t in args.items():
            if not torch.is_tensor(t) or name == "ws":
                continue
            wrong = [t.to(torch.float64)]
            if t.dim() == 2 and name != "logits" and t.shape[1] > 1:
                wrong.append(t.t().contiguous().t())
            if name != "refs" and (name != "pairs" or fn is nt.nt_page_extend):  # these may have any number of entries
                wrong.append(torch.cat((t, t[:1])) if t.numel() > 1 else t[:0])
            for w in wrong:
                with pytest.raises(nt.NtError) as e:
                    fn(**{**args, name: w}, stream=0)
                assert "CUDA" not in str(e.value), (fn.__name__, name, w.shape, str(e.value))
    with pytest.raises(nt.NtError, match="one \\[Hkv, t_stride, D\\] cache per layer"):
        nt.nt_page_copy(caches, nt.pointer_array([k]), 2, 64, 64, 16, z(3, 2))
    with pytest.raises(nt.NtError, match="int range"):
        nt.nt_page_fork(**{**calls[0][1], "page": 1 << 40}, stream=0)


def test_plain_forms_agree_with_a_list_of_lists():
    """The tests' own oracle: every sequence's rows keep what was appended to them."""
    rs = np.random.RandomState(0)
    page, S = 16, 6
    table, length, refs = np.full((S, 6), -1, dtype=np.int32), np.zeros(S, dtype=np.int32), np.zeros(40, dtype=np.int32)
    pool = np.zeros(40 * page, dtype=int)
    lines = [[] for _ in range(S)]
    for t in range(70):
        parent = rs.randint(0, S, S)
        table, length, refs = _paged.fork(table, length, parent, refs, page)
        table, length, refs, rows, pos, pairs, bad = _paged.extend(table, length, refs, [1] * S, page)
        assert bad == 0
        for a, b in pairs:
            if a >= 0:
                pool[b * page:(b + 1) * page] = pool[a * page:(a + 1) * page]
        new = rs.randint(1, 1000, S)
        pool[rows] = new
        lines = [lines[p] + [x] for p, x in zip(parent, new)]
        for s in range(S):
            assert pool[_paged.rows_of(table[s], length[s], page)].tolist() == lines[s]
        if t % 20 == 19:
            refs, table, moves, used = _paged.compact(refs, table, length, page)
            for a, b in moves:
                pool[b * page:(b + 1) * page] = pool[a * page:(a + 1) * page]
            assert (refs[:used] > 0).all() and (refs[used:] == 0).all()
