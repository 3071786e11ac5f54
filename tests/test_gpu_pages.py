"""Bookkeeping of the paged cache on the GPU against the plain forms: whole numbers, which have to be equal."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests import _paged
from tests._gpu import DEV, dev, host

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ints(a):
    return dev(np.ascontiguousarray(a, dtype=np.int32))


def empty(*shape):
    return torch.full(shape, -77, dtype=I32, device=DEV)


def run_fork(table, length, parent, refs, page):
    to, lo, r, bad = empty(len(parent), table.shape[1]), empty(len(parent)), ints(refs), torch.zeros(1, dtype=I32, device=DEV)
    nt.nt_page_fork(ints(table), ints(length), ints(parent), r, page, to, lo, n_bad=bad)
    return host(to), host(lo), host(r), int(bad)


def run_extend(table, length, refs, counts, page, T=None, q_start=None):
    start = np.concatenate(([0], np.cumsum(counts))) if q_start is None else q_start
    T = T or int(max(start[-1], 1))
    t, n, r, rows, pos, pairs = ints(table), ints(length), ints(refs), empty(T), empty(T), empty(len(length), 2)
    bad = torch.zeros(1, dtype=I32, device=DEV)
    nt.nt_page_extend(t, n, r, ints(start), page, rows, pos, pairs, n_bad=bad)
    return [host(x) for x in (t, n, r, rows, pos, pairs)] + [int(bad)]


def check_extend(table, length, refs, counts, page, T=None):
    got = run_extend(table, length, refs, counts, page, T)
    want = _paged.extend(table, length, refs, counts, page)
    n = sum(counts)
    for name, g, w in zip(("table", "length", "refs", "rows", "pos", "pairs"), got, want):
        if name in ("rows", "pos"):
            assert np.array_equal(g[:n], w), (name, g[:n], w)
            assert (g[n:] == (-1 if name == "rows" else 0)).all() or n == len(g) == 0
        else:
            assert np.array_equal(g, w), (name, g, w)
    assert got[6] == want[6]
    return want


def shared_state(rs, S, page, most, n_extra=6):
    """Sequences of which some have been forked from others."""
    lengths = rs.randint(0, most, S)
    table, length, refs = _paged.pool_state(rs, lengths.tolist(), page, spare=n_extra, width=most // page + 6)
    return _paged.fork(table, length, rs.randint(-1, S, S), refs, page)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("S,So", [(1, 1), (1, 8), (8, 8), (7, 3), (300, 300), (4096, 4096)])
def test_fork(S, So, page):
    rs = np.random.RandomState(S + page)
    table, length, refs = _paged.pool_state(rs, rs.randint(0, 5 * page, S).tolist(), page)
    parent = rs.randint(-1, S, So)
    got = run_fork(table, length, parent, refs, page)
    for g, w in zip(got, _paged.fork(table, length, parent, refs, page)):
        assert np.array_equal(g, w)
    assert got[3] == 0


def test_fork_counts_what_is_out_of_range():
    rs = np.random.RandomState(0)
    table, length, refs = _paged.pool_state(rs, [40, 20, 0], 16)
    table[0, 1] = len(refs)
    table[1, 1] = -5
    table[2, 0] = 1 << 30  # not in use
    got = run_fork(table, length, np.array([0, 1, 3, -2, 2]), refs, 16)
    assert got[3] == 2 + 2 and list(got[1]) == [40, 20, 0, 0, 0]
    assert np.array_equal(got[2], refs)  # one child each, and nothing out of range
    assert np.array_equal(got[0][0][:3], table[0][:3]) and (got[0][2:] == -1).all()
    long = np.array([10 ** 9], dtype=np.int32)
    assert run_fork(table[:1], long, np.array([0]), refs, 16)[1][0] == table.shape[1] * 16


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("S", [1, 2, 8, 33, 500])
@pytest.mark.parametrize("kind", ["token", "ragged", "prompt"])
def test_extend(S, page, kind):
    rs = np.random.RandomState(S + page)
    counts = {"token": [1] * S, "ragged": rs.randint(0, 3 * page, S).tolist(),
              "prompt": (rs.randint(0, 2, S) * rs.randint(1, 2 * page, S)).tolist()}[kind]
    table, length, refs = shared_state(rs, S, page, 3 * page, n_extra=S + sum(_paged.pages_of(c, page) + 1 for c in counts))
    check_extend(table, length, refs, counts, page, T=max(1, sum(counts)) + rs.randint(0, 9))


def test_extend_many_sequences_and_a_large_pool():
    rs = np.random.RandomState(3)
    table, length, refs = shared_state(rs, 4096, 16, 30, n_extra=20000)
    check_extend(table, length, refs, [1] * 4096, 16)


@pytest.mark.parametrize("shift", [0, 1, 3])
def test_extend_counts_at_any_alignment(shift):
    rs = np.random.RandomState(5)
    table, length, refs = shared_state(rs, 20, 16, 60, n_extra=8200)
    big = torch.zeros(len(refs) + 4, dtype=I32, device=DEV)
    r = big[shift:shift + len(refs)]
    r.copy_(ints(refs))
    t, n, rows, pos, pairs = ints(table), ints(length), empty(20), empty(20), empty(20, 2)
    nt.nt_page_extend(t, n, r, ints(np.arange(21)), 16, rows, pos, pairs)
    want = _paged.extend(table, length, refs, [1] * 20, 16)
    for g, w in zip((t, n, r, rows, pos, pairs), want):
        assert np.array_equal(host(g), w)


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 7])
def test_extend_when_the_pages_run_out(spare):
    rs = np.random.RandomState(spare)
    table, length, refs = shared_state(rs, 12, 16, 50, n_extra=0)
    free = np.flatnonzero(refs == 0)
    refs[free[spare:]] = 1  # held by someone else
    want = check_extend(table, length, refs, [1, 20, 0, 3, 16, 1, 0, 40, 2, 2, 1, 5], 16)
    assert spare > 6 or want[6] > 0


def test_extend_leaves_what_cannot_be_extended():
    page = 16
    table = np.array([[0, 1], [2, 3], [4, -1], [99, -1], [5, 6]], dtype=np.int32)
    length = np.array([32, 20, -3, 5, 17], dtype=np.int32)  # full, fine, negative, a bad last page, fine
    refs = np.array([1, 1, 1, 1, 1, 1, 1, 0, 0, 0, 0], dtype=np.int32)
    want = check_extend(table, length, refs, [1, 2, 1, 1, 2], page)
    assert want[6] == 3


def test_extend_starts_out_of_range_are_cut():
    table, length, refs = _paged.pool_state(np.random.RandomState(0), [5, 5], 16)
    got = run_extend(table, length, refs, None, 16, T=6, q_start=np.array([-4, 3, 100]))
    want = _paged.extend(table, length, refs, [3, 3], 16)
    assert all(np.array_equal(g, w) for g, w in zip(got[:6], want))


@pytest.mark.parametrize("n,S", [(1, 1), (2, 1), (300, 7), (1024, 3), (5001, 60), (20000, 500)])
@pytest.mark.parametrize("used", [0.0, 0.1, 0.6, 1.0])
def test_compact(n, S, used):
    rs = np.random.RandomState(n + S)
    ids = rs.permutation(n)[:int(n * used)]
    held = np.bincount(rs.randint(0, S, len(ids)), minlength=S)
    table = np.full((S, int(held.max()) + 2), -1, dtype=np.int32)
    at = 0
    for s in range(S):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    refs = np.bincount(ids, minlength=n).astype(np.int32)
    refs[refs > 0] += rs.randint(0, 4, int((refs > 0).sum())).astype(np.int32)
    length = np.maximum(held * 16 - rs.randint(0, 16, S), 0).astype(np.int32)
    for s in range(S):  # entries that are not in use
        table[s, _paged.pages_of(length[s], 16):] = rs.randint(0, n)
    r, t, pairs, used_out = ints(refs), ints(table), empty(n // 2 + 3, 2), empty(1)
    ws = torch.zeros(nt.nt_page_compact_workspace_size(n), dtype=torch.uint8, device=DEV)
    bad = torch.zeros(1, dtype=I32, device=DEV)
    nt.nt_page_compact(r, t, ints(length), 16, pairs, used_out, ws, n_bad=bad)
    want = _paged.compact(refs, table, length, 16)
    assert np.array_equal(host(r), want[0]) and np.array_equal(host(t), want[1])
    m = len(want[2])
    assert np.array_equal(host(pairs)[:m], want[2]) and (host(pairs)[m:] == -1).all()
    assert int(used_out) == want[3] and int(bad) == 0


@pytest.mark.parametrize("L,Hkv,D,page", [(1, 1, 8, 16), (3, 2, 64, 16), (2, 5, 128, 64), (130, 1, 16, 16), (1, 3, 256, 256), (2, 2, 24, 32)])
@pytest.mark.parametrize("n", [1, 5, 40])
def test_copy(L, Hkv, D, page, n):
    rs = np.random.RandomState(n + D)
    n_pages = 2 * n + 3
    ts = n_pages * page + 5  # rows behind the last page
    caches = [torch.randint(-30000, 30000, (2, Hkv, ts, D), device=DEV, dtype=torch.int16).view(torch.bfloat16) for _ in range(L)]
    ids = rs.permutation(n_pages)
    pairs = np.stack((ids[:n], ids[n:2 * n]), 1)
    some = rs.uniform(size=n) < 0.6
    skip = [(-1, -1), (n_pages, 1), (0, -3), (-1, 2)]
    for i in np.flatnonzero(~some):
        pairs[i] = skip[i % 4]
    want = [c.clone() for c in caches]
    for w in want:
        for a, b in pairs[some]:
            w[:, :, b * page:(b + 1) * page] = w[:, :, a * page:(a + 1) * page]
    k, v = nt.pointer_array([c[0] for c in caches]), nt.pointer_array([c[1] for c in caches])
    nt.nt_page_copy(k, v, Hkv, D, ts, page, ints(pairs))
    for c, w in zip(caches, want):
        assert torch.equal(c.view(torch.int16), w.view(torch.int16))


def test_copy_more_pairs_than_a_round_holds():
    n, page = 2500, 16
    cache = torch.randn(2, 1, 2 * n * page, 8, device=DEV).bfloat16()
    ids = np.random.RandomState(0).permutation(2 * n)
    pairs = np.stack((ids[:n], ids[n:]), 1)
    want = cache.clone().view(2, 1, 2 * n, page * 8)
    want[:, :, ids[n:]] = want[:, :, ids[:n]]
    nt.nt_page_copy(nt.pointer_array([cache[0]]), nt.pointer_array([cache[1]]), 1, 8, 2 * n * page, page, ints(pairs))
    assert torch.equal(cache, want.view_as(cache))


@pytest.mark.parametrize("graph", [False, True])
def test_steps_of_beams(graph):
    """Fork, extend and copy for many steps, on a stream of their own and in a replayed graph: every sequence's rows are those of its
    line of ancestors, and the counts those of its pages."""
    rs = np.random.RandomState(1)
    S, page, L, Hkv, D, n_pages = 9, 16, 2, 1, 8, 80
    ts = n_pages * page
    tables, lengths, refs = [empty(S, 7), empty(S, 7)], [torch.zeros(S, dtype=I32, device=DEV) for _ in range(2)], torch.zeros(n_pages, dtype=I32, device=DEV)
    parent, start = torch.zeros(S, dtype=I32, device=DEV), ints(np.arange(S + 1))
    rows, pos, pairs = empty(S), empty(S), empty(S, 2)
    caches = [torch.zeros(2, Hkv, ts, D, dtype=torch.bfloat16, device=DEV) for _ in range(L)]
    k, v = nt.pointer_array([c[0] for c in caches]), nt.pointer_array([c[1] for c in caches])
    new = torch.zeros(S, Hkv, D, device=DEV)
    q = torch.zeros(S, Hkv, D, device=DEV)

    def step():
        nt.nt_page_fork(tables[0], lengths[0], parent, refs, page, tables[1], lengths[1])
        nt.nt_page_extend(tables[1], lengths[1], refs, start, page, rows, pos, pairs)
        nt.nt_page_copy(k, v, Hkv, D, ts, page, pairs)
        for c in caches:
            nt.nt_qk_norm_rope_append(q, new, new, None, None, 1e-6, None, nt.NT_ROPE_HALF, 1.0, q, c[0], c[1], pos=pos, rows=rows)
        tables[0].copy_(tables[1])
        lengths[0].copy_(lengths[1])

    stream = torch.cuda.Stream()
    g = None
    lines = [[] for _ in range(S)]
    with torch.cuda.stream(stream):
        for t in range(90):
            up = rs.randint(0, S, S) if t % 3 else np.arange(S)
            if t % 10 == 9:
                up[rs.randint(0, S)] = -1
            values = rs.randint(1, 200, S)
            parent.copy_(ints(up))
            new.copy_(dev(values.astype(np.float32))[:, None, None].expand(S, Hkv, D))
            if graph and t == 5:
                stream.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    step()
            g.replay() if g else step()
            lines = [(lines[p] if p >= 0 else []) + [x] for p, x in zip(up, values)]
            stream.synchronize()
            tb, ln, rf = host(tables[0]), host(lengths[0]), host(refs)
            assert ln.tolist() == [len(x) for x in lines]
            count = np.zeros(n_pages, dtype=int)
            for s in range(S):
                np.add.at(count, tb[s, :_paged.pages_of(ln[s], page)], 1)
            assert np.array_equal(count, rf)
            for c in caches:
                c = host(c.float())
                for s in range(S):
                    at = _paged.rows_of(tb[s], ln[s], page)
                    assert (c[:, 0, at, :] == np.array(lines[s])[None, :, None]).all()
            if max(ln) > 100:
                break
