"""Weights of chunks of fp32 queries with heads of 64 are fp32: nothing is lost in the terms they are multiplied in."""
import pytest
import torch

from tests import _paged
from tests.test_gpu_paged_attention import DEV, U32, Call
from tests.test_gpu_paged_weights import SPAN, shares, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,new", [(1, 1, 9), (4, 1, 16), (16, 2, 3), (64, 1, 2), (8, 2, 30)])
@pytest.mark.parametrize("length", [7, 20, 33])
def test_weights_keep_24_bits(length, Hq, Hkv, new):
    """As for few rows: queries of 0, values of one 1 each. A weight's terms are added in three k-steps (every other one adds nothing to its
    sum), each cut off by 2^-23 at most: 6 of 2^-24 in place of 4."""
    rows = length + new
    c = Call(f"{new}+{length}", Hq, Hkv, 64, 16, "f32", seed=length)
    c.q = torch.zeros_like(c.q)
    c.slopes = slopes_of(Hq, rows)
    at = torch.from_numpy(_paged.rows_of(c.table[0], rows, 16)).to(DEV)
    c.v[:, at] = torch.eye(rows, 64, device=DEV).bfloat16()
    got = shares(c.run().double())
    want = shares(_paged.attend(c.q, c.k, c.v, c.table, c.counts, c.length, c.page, slopes=c.slopes)[0])
    T = SPAN * 1.4427
    worst = float(((got - want).abs() / want.clamp(min=1e-9))[want > 0].max())
    assert worst <= 2 * (0.6932 * 4 * T + 4 + 6 + 3) * U32, worst / U32
