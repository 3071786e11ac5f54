"""A pool of one page, whose compaction has no pairs: the header's n >= n_pages / 2 is 0 there."""
import pytest
import torch

from packed_weight_gemv_gb300 import build as nt_build
from packed_weight_gemv_gb300 import nt
from tests.test_pages_cpu import COMPACT
from tests.test_tree_cpu import INV, call, reaches_device


@pytest.fixture(scope="module")
def lib():
    nt_build.build()
    return nt.load_library()


def test_compaction_without_pairs(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real: only where there is no device")
    assert reaches_device(call(lib.nt_page_compact, COMPACT, n=1, m=0, pairs=None))
    assert call(lib.nt_page_compact, COMPACT, n=2, m=0, pairs=None) == INV
    assert call(lib.nt_page_compact, COMPACT, n=1, m=1, pairs=None) == INV
