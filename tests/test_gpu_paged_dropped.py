"""Pages that a window has left behind: a server may drop them (-1 in the table) and reuse them. They are no bad entries, and nothing of
them is read; an entry out of range among the rows that are seen still counts."""
import numpy as np
import pytest
import torch

from tests import _paged
from tests._gpu import DEV
from tests.test_gpu_paged_attention import Call, ints

pytestmark = pytest.mark.gpu
SEQS = ["1+300", "1+1000 1+70 1+513", "3+200 1+90", "40+200", "150+333 1+700", "300+500 20+129"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("window", [1, 17, 50, 100, 130, 255])
@pytest.mark.parametrize("seqs", SEQS)
def test_dropped_pages(seqs, window, page, dtype):
    c = Call(seqs, 4, 2, 64, page, dtype, window=window, seed=window)
    n_bad = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = c.run(n_bad=n_bad)
    c.check(want)
    assert int(n_bad) == 0
    table = c.table.copy()
    dropped = 0
    for s, n in enumerate(c.counts):
        last = max(0, int(c.length[s]) - n - window + 1) // page  # the page of the lowest row that is seen
        table[s, :last] = np.resize([-1, 1 << 28, -(1 << 31)], last)
        dropped += last
    assert dropped > 0 or page > 16 or window > 50
    out = c.run(n_bad=n_bad, table=ints(table))
    assert int(n_bad) == 0, "pages that nobody sees"
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window", [17, 100])
@pytest.mark.parametrize("seqs", SEQS)
def test_the_page_of_the_lowest_row_that_is_seen_counts(seqs, window, dtype):
    c = Call(seqs, 4, 2, 64, 16, dtype, window=window)
    for s, n in enumerate(c.counts):
        first = max(0, int(c.length[s]) - n - window + 1) // 16
        table = c.table.copy()
        table[s, first] = -1
        n_bad = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = c.run(n_bad=n_bad, table=ints(table))
        assert int(n_bad) > 0
        keep = c.k.clone(), c.v.clone()
        rows = _paged.rows_of(c.table[s], min(int(c.length[s]), 16 * first + 16), 16)[16 * first:]
        c.k[:, rows], c.v[:, rows] = 0.0, 0.0
        c.check(out)
        c.k, c.v = keep
