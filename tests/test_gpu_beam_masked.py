"""Beams whose logits are masked by the type's lowest value, and logits near the ends of the range."""
import numpy as np
import pytest

from tests.test_gpu_beam import random, run

pytestmark = pytest.mark.gpu
LOW = np.finfo(np.float32).min


def chosen(x, scores, W, K, alpha=0.0, lengths=None):
    """parent, token and score in 64 bits with the largest logit taken off first, so that the largest ones cost the others nothing."""
    parent, token, score = [], [], []
    for g in range(len(x) // W):
        cand = []
        for b in range(g * W, (g + 1) * W):
            d = x[b].astype(np.float64) - float(x[b].max())
            total = (float(scores[b]) - np.log(np.exp(d).sum())) + d
            rank = total / (int(lengths[b]) + 1.0) ** alpha if alpha else total
            # (within a beam by the logits themselves: next to a score of -3e38 even 64 bits lose them)
            for v in np.lexsort((np.arange(len(d)), -d, -rank))[:K]:
                if total[v] >= LOW:  # (what leaves the range counts as -inf)
                    cand.append((rank[v], b, int(v), total[v]))
        cand.sort(key=lambda c: (-c[0], c[1]))  # (stable: a beam's own stay in order)
        cand = cand[:K] + [(0, -1, -1, -np.inf)] * (K - len(cand[:K]))
        parent += [c[1] for c in cand]
        token += [c[2] for c in cand]
        score += [c[3] for c in cand]
    return np.array(parent), np.array(token), np.array(score)


def check(x, scores, W, K, **kw):
    got, want = run(x, scores, W, K, **kw), chosen(x, scores, W, K, **kw)
    assert np.array_equal(got[0], want[0]), (got[0], want[0])
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    there = want[0] >= 0
    # the header's bound, with logits less their row's largest: what is far below it does not enter
    assert (np.abs(got[2][there] - want[2][there]) <= 2.0 ** -22 * np.maximum(np.abs(want[2][there]), 1.0)).all(), (got[2], want[2])
    assert (got[2][~there] == -np.inf).all()
    return got


@pytest.mark.parametrize("alpha", [0.0, 0.7])
@pytest.mark.parametrize("fill", [LOW, -1e38, -1e30, 3e38])
@pytest.mark.parametrize("V", [40, 3001])
def test_a_row_that_is_masked_altogether_has_the_chance_of_any_token(V, fill, alpha):
    """All logits alike: each is -log V, wherever they stand. Such a beam must not overtake the others."""
    x, s = random(np.random.RandomState(V), 8, V)
    x[1], x[6] = fill, fill
    s[6] = -1000.0
    check(x, s, 4, 6, alpha=alpha, lengths=np.arange(8) * 3 if alpha else None)


@pytest.mark.parametrize("V", [40, 3001])
def test_few_tokens_left_by_a_mask(V):
    x, s = random(np.random.RandomState(V + 1), 6, V)
    keep = x[:, [3, V - 1]].copy()
    x[:] = LOW
    x[:, [3, V - 1]] = keep
    got = check(x, s, 3, 6)
    assert set(got[1].tolist()) == {3, V - 1}


@pytest.mark.parametrize("V", [40, 3001])
def test_differences_that_leave_the_range(V):
    """The best of a row near the largest number, the rest near the lowest: those have no chance, and are not chosen before others."""
    x, s = random(np.random.RandomState(V + 2), 6, V)
    x[0] = LOW
    x[0, 7] = 3e38
    x[4] = -3e38
    x[4, 11], x[4, 12] = 3.2e38, 3.2e38
    check(x, s, 3, 5)
    x[1:3] = -np.inf
    x[1:3, 0] = [1.0, 2.0]
    got = run(x, s, 3, 5)
    assert got[0][:5].tolist().count(-1) == 2 and sorted(got[0][:3].tolist()) == [0, 1, 2]


def test_scores_near_the_end_of_the_range():
    x, s = random(np.random.RandomState(3), 4, 500)
    s[:] = [-3.4e38, -3e38, -1.0, -2.0]
    check(x, s, 2, 4)
    check(x, s, 4, 4)
