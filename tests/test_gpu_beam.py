"""Beam selection on the GPU against 64 bits: parents and tokens are equal, scores within 2^-22 of the larger of score and
logits (the header's bound: fp32 roundings of the chunks' sums and of the result)."""
import numpy as np
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests import _paged
from tests._gpu import DEV, dev, host

pytestmark = pytest.mark.gpu


def run(logits, scores, W, K, done=None, eos=-1, lengths=None, alpha=0.0, ws=None):
    N, V = logits.shape
    out = [torch.full((N // W * K,), -77, dtype=torch.int32, device=DEV) for _ in range(3)]
    score = torch.full((N // W * K,), float("nan"), device=DEV)
    ws = torch.zeros(nt.nt_beam_select_workspace_size(V, N), dtype=torch.uint8, device=DEV) if ws is None else ws
    t = lambda a: None if a is None else dev(np.asarray(a, dtype=np.int32))  # noqa: E731
    x = logits if torch.is_tensor(logits) else dev(logits.astype(np.float32))
    nt.nt_beam_select(x, dev(np.asarray(scores, dtype=np.float32)), W, out[0], out[1], score, ws, done=t(done), done_out=out[2], eos=eos,
                      lengths=t(lengths), alpha=alpha)
    return host(out[0]), host(out[1]), host(score), host(out[2])


def check(logits, scores, W, K, done=None, eos=-1, lengths=None, alpha=0.0):
    got = run(logits, scores, W, K, done, eos, lengths, alpha)
    want = _paged.beam(logits, np.asarray(scores, dtype=np.float32), W, K, done, eos, lengths, alpha)
    assert np.array_equal(got[0], want[0]), (got[0], want[0])
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[3], want[3])
    there = want[0] >= 0
    size = np.abs(logits[np.isfinite(logits)]).max(initial=0.0)
    err = np.abs(got[2][there] - want[2][there])
    assert (err <= 2.0 ** -22 * np.maximum(np.abs(want[2][there]), max(size, 1.0))).all(), err.max()
    assert (got[2][~there] == -np.inf).all()
    return got


def random(rs, N, V, spread=2.0):
    x = rs.randn(N, V) * spread
    x[np.arange(N)[:, None], rs.randint(0, V, (N, 5))] += 7.0
    return x.astype(np.float32), (-10 * rs.rand(N)).astype(np.float32)


@pytest.mark.parametrize("G,W,K,V", [(1, 1, 1, 1), (1, 1, 3, 2), (2, 1, 1, 1000), (3, 4, 4, 511), (3, 4, 8, 512), (2, 5, 5, 513),
                                     (1, 16, 32, 4099), (2, 64, 64, 1500), (5, 3, 64, 2048), (1, 2, 64, 20), (1, 4, 4, 151936),
                                     (2, 8, 8, 32003), (1, 2, 7, 300001)])
def test_select(G, W, K, V):
    rs = np.random.RandomState(V + W)
    check(*random(rs, G * W, V), W, K)


@pytest.mark.parametrize("alpha", [0.0, 0.6, 1.0, 2.5])
@pytest.mark.parametrize("W,K,V", [(1, 2, 700), (4, 4, 1003), (12, 24, 5000), (33, 50, 600)])
def test_finished_beams_and_lengths(W, K, V, alpha):
    rs = np.random.RandomState(W + V)
    x, s = random(rs, 3 * W, V)
    done = (rs.rand(3 * W) < 0.4).astype(np.int32)
    done[W:2 * W] = 1  # a group that has ended
    lengths = rs.randint(0, 50, 3 * W)
    got = check(x, s, W, K, done, V // 2, lengths, alpha)
    assert (got[3][K:K + min(W, K)] == 1).all()


@pytest.mark.parametrize("alpha", [1.0, 4.0])
@pytest.mark.parametrize("most", [300, 1 << 20, (1 << 31) - 1])
def test_steep_penalties_of_long_beams(alpha, most):
    """1 / length^alpha is 2^-124 at the smallest, so it ranks every beam; scores are not touched by it."""
    rs = np.random.RandomState(most & 0xffff)
    x, s = random(rs, 8, 900)
    check(x, s, 4, 6, np.array([0, 1, 0, 0] * 2), 7, rs.randint(most // 2, most, 8), alpha)


def test_ties_go_to_the_lower_beam_and_token():
    V = 3001
    for fill in (0.0, -3.25, 1e-30):
        x = np.full((8, V), fill, dtype=np.float32)
        got = check(x, np.zeros(8), 4, 8)
        assert got[0].tolist() == [0] * 8 + [4] * 8 and got[1].tolist() == list(range(8)) * 2
    x = np.zeros((4, V), dtype=np.float32)
    x[:, [2999, 17, 512, 511, 1024]] = 4.0
    got = check(x, np.zeros(4), 4, 20)
    assert got[1].tolist() == [17, 511, 512, 1024, 2999] * 4
    assert got[0].tolist() == [0] * 5 + [1] * 5 + [2] * 5 + [3] * 5


def test_more_alike_than_the_list_holds():
    """Thousands of equal values that straddle chunks, with a few above them."""
    rs = np.random.RandomState(2)
    x = np.where(rs.rand(6, 9000) < 0.5, 1.0, -5.0).astype(np.float32)
    x[3, 8000], x[5, 3] = 2.0, 3.0
    for K in (1, 2, 9, 64):
        check(x, np.zeros(6), 3, K)
        check(x, [-1, 0, -1, 0, 0, 0], 6, K)


def test_infinities_and_nans():
    rs = np.random.RandomState(4)
    x, s = random(rs, 12, 2000)
    x[0] = -np.inf                       # nothing allowed
    x[1, ::2] = np.nan
    x[2, 5] = np.inf                     # no continuation
    x[4, 700:] = -np.inf
    x[5] = np.nan
    x[6:9] = -np.inf                     # a group without any
    x[6, 1999] = 2.0                     # but one
    s[9], s[10] = -np.inf, np.nan
    got = check(x, s, 3, 6)
    assert got[0][12:18].tolist() == [6, -1, -1, -1, -1, -1]
    x[:] = -np.inf
    got = check(x, s, 3, 6)
    assert (got[0] == -1).all()


def test_close_continuations_of_different_beams():
    """Scores far from 0 whose sums with the logits differ by less than a step of fp32 at their size."""
    V = 4000
    x = np.full((2, V), -30.0, dtype=np.float32)
    x[0, 100], x[1, 7] = 5.0, 5.0
    x[1, 8] = np.nextafter(np.float32(5.0), np.float32(6.0))
    x[0, 101] = np.nextafter(x[1, 8], np.float32(6.0))
    got = check(x, [-1000.0, -1000.0], 2, 4)
    assert set(zip(got[0].tolist(), got[1].tolist())) == {(0, 100), (0, 101), (1, 7), (1, 8)}


def test_large_logits():
    rs = np.random.RandomState(7)
    x, s = random(rs, 4, 3000, spread=1e4)
    check(x, s, 4, 4)
    x, s = random(rs, 4, 3000, spread=1e-4)
    check(x * np.float32(1e-3), s, 4, 16)


def test_rows_at_any_alignment_and_one_workspace_for_many_calls():
    rs = np.random.RandomState(8)
    ws = torch.zeros(nt.nt_beam_select_workspace_size(5000, 8), dtype=torch.uint8, device=DEV)
    for V in (4996, 4997, 4998, 5000):
        x, s = random(rs, 8, V)
        big = torch.zeros(8 * V + 3, device=DEV)
        for shift in (0, 1, 2, 3):
            y = big[shift:shift + 8 * V].view(8, V)
            y.copy_(dev(x))
            got = run(y, s, 4, 4, ws=ws)
            want = _paged.beam(x, s, 4, 4)
            assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    x[4:] = x[:4]  # the same group twice gives the same bits
    s[4:] = s[:4]
    got = run(x, s, 4, 4, ws=ws)
    assert np.array_equal(got[1][:4], got[1][4:]) and np.array_equal(got[2][:4], got[2][4:])


def test_in_a_graph_on_another_stream():
    rs = np.random.RandomState(9)
    x, s = random(rs, 8, 6001)
    logits, scores = dev(x), dev(s)
    out = [torch.zeros(8, dtype=torch.int32, device=DEV) for _ in range(2)]
    score = torch.zeros(8, device=DEV)
    ws = torch.zeros(nt.nt_beam_select_workspace_size(6001, 8), dtype=torch.uint8, device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step = lambda: nt.nt_beam_select(logits, scores, 4, out[0], out[1], score, ws)  # noqa: E731
        step()
        stream.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            step()
        for _ in range(5):
            x, s = random(rs, 8, 6001)
            logits.copy_(dev(x))
            scores.copy_(dev(s))
            g.replay()
            stream.synchronize()
            want = _paged.beam(x, s, 4, 4)
            assert np.array_equal(host(out[0]), want[0]) and np.array_equal(host(out[1]), want[1])
