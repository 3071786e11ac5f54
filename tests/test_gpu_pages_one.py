"""A pool of one page: compaction and the copy behind it take no pairs."""
import pytest
import torch

from packed_weight_gemv_gb300 import nt
from tests._gpu import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("used", [0, 1])
def test_compaction_and_copy(used):
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    refs, table, length, n_used = i32(used), i32(0).view(1, 1), i32(5 * used), i32(-7)
    pairs = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    ws = torch.zeros(nt.nt_page_compact_workspace_size(1), dtype=torch.uint8, device=DEV)
    cache = torch.randn(2, 1, 16, 64, device=DEV).bfloat16()
    want = cache.clone()
    nt.nt_page_compact(refs, table, length, 16, pairs, n_used, ws)
    nt.nt_page_copy(nt.pointer_array([cache[0]]), nt.pointer_array([cache[1]]), 1, 64, 16, 16, pairs)
    assert n_used.tolist() == [used] and refs.tolist() == [used] and table.tolist() == [[0]] and torch.equal(cache, want)
