"""Weights of fp32 queries with few rows are fp32: nothing is lost in the terms they are multiplied in."""
import pytest
import torch

from tests import _paged
from tests.test_gpu_paged_attention import DEV, U32, Call

pytestmark = pytest.mark.gpu
SPAN = 0.7  # scores lie this far apart at most


def shares(out):
    """Of each value among those of a row: what is common to all (the sum of the weights, its inverse) leaves no trace."""
    return out / out.sum(-1, keepdim=True)


def slopes_of(Hq, rows):
    return SPAN / rows * (torch.arange(Hq, device=DEV) + 1.0) / Hq


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,new", [(1, 1, 1), (4, 1, 1), (2, 2, 3), (5, 1, 1), (8, 1, 1), (12, 2, 1), (2, 1, 4), (4, 4, 8)])
@pytest.mark.parametrize("length", [7, 20, 40, 55])
def test_weights_keep_24_bits(length, Hq, Hkv, new, D):
    """Queries of 0 and values of one 1 each, so that an output is a weight: scores are the bias alone. With T = SPAN log2 e, a weight
    2^(x log2 e - m) has the bias' rounding, the products' (log2 e is rounded as well) and the difference's, 4 T of 2^-24 in the exponent, ln 2 of that in
    the weight, and ex2.approx 2^-22; its terms' sum 4 and the output 3 of 2^-24. A share has twice that. Weights of two rounded bf16 terms are off by up to
    2^-17, 128 of 2^-24 (in these cases by 62 to 113)."""
    rows = length + new
    c = Call(f"{new}+{length}", Hq, Hkv, D, 16, "f32", seed=length)
    c.q = torch.zeros_like(c.q)
    c.slopes = slopes_of(Hq, rows)
    at = torch.from_numpy(_paged.rows_of(c.table[0], rows, 16)).to(DEV)
    c.v[:, at] = torch.eye(rows, D, device=DEV).bfloat16()
    got = shares(c.run().double())
    want = shares(_paged.attend(c.q, c.k, c.v, c.table, c.counts, c.length, c.page, slopes=c.slopes)[0])
    T = SPAN * 1.4427
    worst = float(((got - want).abs() / want.clamp(min=1e-9)).max())
    assert worst <= 2 * (0.6932 * 4 * T + 4 + 4 + 3) * U32, worst / U32
