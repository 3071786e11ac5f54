"""Lists of pairs whose indexes would leave the int range are refused on the host."""
import pytest
import torch

from packed_weight_gemv_gb300 import build as nt_build
from packed_weight_gemv_gb300 import nt
from tests.test_pages_cpu import COMPACT, copy_args
from tests.test_tree_cpu import INV, call, reaches_device


@pytest.fixture(scope="module")
def lib():
    nt_build.build()
    return nt.load_library()


@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - 1])
def test_long_lists_are_refused(lib, n):
    assert call(lib.nt_page_copy, copy_args(n=n)) == INV
    assert call(lib.nt_page_compact, COMPACT, m=n) == INV


def test_the_longest_lists_are_not(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real: only where there is no device")
    assert reaches_device(call(lib.nt_page_copy, copy_args(n=1 << 30)))
    assert reaches_device(call(lib.nt_page_compact, COMPACT, m=1 << 30))
