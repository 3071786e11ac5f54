"""Beam selection where there are hardly more chunks than results: small vocabularies with many beams, finished beams, and best
continuations that stand in few threads' hands."""
import numpy as np
import pytest

from tests.test_gpu_beam import check, random

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("done", [0.0, 0.3, 0.9])
@pytest.mark.parametrize("W,K,V", [(16, 32, 1000), (32, 64, 1000), (32, 64, 1500), (16, 32, 2000), (64, 64, 511), (64, 64, 512), (1, 64, 1000), (1, 64, 32767),
                                   (2, 64, 1100), (8, 16, 513), (4, 64, 2048), (32, 32, 1023), (3, 64, 300)])
def test_more_continuations_reach_the_bound_than_a_list_holds(W, K, V, done):
    rs = np.random.RandomState(W + V)
    x, _ = random(rs, 2 * W, V)
    s = (-12 * rs.rand(2 * W)).astype(np.float32)
    fin = (rs.rand(2 * W) < done).astype(np.int32)
    check(x, s, W, K, fin, V - 1, rs.randint(0, 30, 2 * W), 0.6)


@pytest.mark.parametrize("K", [1, 31, 64])
@pytest.mark.parametrize("lane", [0, 5, 31])
def test_best_continuations_that_one_lane_holds(lane, K):
    """Every 32nd logit is high: the bound of the threads' best ones lies low, and most of what is above it stands with one of them."""
    rs = np.random.RandomState(lane)
    x = rs.randn(16, 1500).astype(np.float32)
    x[:, lane::32] += 9.0
    check(x, -rs.rand(16).astype(np.float32), 16, K)
    check(x, -rs.rand(16).astype(np.float32), 8, K)


@pytest.mark.parametrize("V", [40, 700])
def test_alike_with_few_chunks(V):
    x = np.zeros((32, V), dtype=np.float32)
    check(x, np.zeros(32), 32, 64)
    x[5:9] = 1.0
    x[7, V // 2] = 1.5
    check(x, -np.arange(32) // 9, 16, 33)
