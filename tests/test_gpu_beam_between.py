"""Order of continuations of different beams: right where they differ by more than the bound that the header states for log-sums."""
import numpy as np
import pytest

from tests.test_gpu_beam import run

pytestmark = pytest.mark.gpu
APART = 2.0 ** -16  # twice the bound: both rows may be off by it


@pytest.mark.parametrize("V", [900, 3001, 151936])
@pytest.mark.parametrize("seed", range(6))
def test_rows_of_different_kinds(seed, V):
    """A peaked row, a flat one and one whose logits are all but the first alike, ten below it; their best continuations as far apart
    as the bound allows, in every order."""
    rs = np.random.RandomState(seed)
    x = np.zeros((3, V), dtype=np.float32)
    x[0] = rs.randn(V) - 20.0
    x[0, rs.randint(V)] = 1.0
    x[1] = rs.randn(V) * 0.5
    x[2] = -10.0 + 0.37 * seed
    x[2, 0] = 0.0
    d = x.astype(np.float64) - x.max(1, keepdims=True)
    best = d.max(1) - np.log(np.exp(d).sum(1))  # of each row, without its score
    order = rs.permutation(3)
    goal = -9.0 - 1.25 * APART * np.arange(3)  # totals, apart by a little more
    scores = np.zeros(3, dtype=np.float32)
    scores[order] = goal - best[order]
    total = scores.astype(np.float64) + best
    assert (np.diff(total[order]) <= -APART).all(), "the roundings of the scores"
    parent, token, score, _ = run(x, scores, 3, 3)
    assert parent.tolist() == order.tolist() and np.array_equal(token, x.argmax(1)[order])
    assert (np.abs(score - total[order]) <= 2.0 ** -22 * 20.0).all()
