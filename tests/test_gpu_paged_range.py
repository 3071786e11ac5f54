"""Scores of -inf and values near the end of the stated range."""
import pytest
import torch

from tests import _paged
from tests.test_gpu_paged_attention import DEV, Call

pytestmark = pytest.mark.gpu
SEQS = ["1+40", "1+700 1+70", "3+100", "70+90", "300+200 1+30"]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", SEQS)
def test_a_score_of_minus_infinity_has_no_weight(seqs, D):
    c = Call(seqs, 4, 2, D, 16, "bf16")
    c.q = c.q.abs() + 0.01
    length = int(c.length[0])
    at = torch.from_numpy(_paged.rows_of(c.table[0], length, 16)).to(DEV)
    # every third key: a query of one sign makes its score -inf, and the value beside it does not enter
    c.k[:, at[::3], 5] = -float("inf")
    out = c.run()
    keep = c.k.clone(), c.v.clone()
    want = []
    for v in (1.0, -50.0):
        c.v[:, at[::3]] = v
        want.append(c.run())
    assert torch.equal(want[0], want[1])
    c.k, c.v = keep
    c.check(out)
    c.k[:, at, 5] = -float("inf")
    out = c.run()
    assert (out[:c.counts[0]] == 0).all() and torch.isfinite(out[:sum(c.counts)]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs", SEQS)
def test_values_up_to_2_64(seqs, dtype):
    """Scores that rise by more than a reference's slack, so that weights reach their largest."""
    c = Call(seqs, 4, 2, 64, 16, dtype, scale=3.0)
    c.v = (c.v.float() * 2.0 ** 61).bfloat16()
    c.check(c.run())
