"""The operators over a cache's pages with as many pages, rows and entries as a handle takes, against tests/pages_ref.py."""

import pytest
import torch

import paged_kv_cache_reshape_gb300 as pa
from test_gpu_pages import check_compact, check_fork, check_resize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    pa.build()


@pytest.mark.parametrize("NB", [100_003, 1 << 20])
def test_pools_of_many_pages(NB):
    g = torch.Generator().manual_seed(NB)
    R, MB, bs = 700, 9, 16
    lengths = torch.randint(0, MB * bs + 1, (R,), generator=g).tolist()
    delta = [int(torch.randint(-x, MB * bs - x + 1, (1,), generator=g)) for x in lengths]
    parent = torch.randint(-1, R, (900,), generator=g).tolist()

    def low_pages_used(table, ref, *_):  # fresh pages are far up, and compaction moves from there
        for p in range(NB - 5000):
            ref[p] = max(ref[p], int(p % 3000 != 7))

    check_fork(R, MB, bs, lengths, NB, parent, 16, 1, change=low_pages_used)
    check_resize(R, MB, bs, lengths, NB, delta, 16, 1, change=low_pages_used)
    check_compact(R, MB, bs, lengths, NB, 16, 1)
    check_compact(R, MB, bs, lengths, NB, 16, 1, change=low_pages_used)


def test_many_rows():
    """Rows and children by the hundred thousand, of one page at most."""
    g = torch.Generator().manual_seed(1)
    R, bs, NB = 100_000, 16, 250_000
    lengths = torch.randint(0, bs + 1, (R,), generator=g).tolist()
    delta = (torch.randint(0, bs + 1, (R,), generator=g) - torch.tensor(lengths)).tolist()
    parent = torch.randint(-1, R, (R + 77,), generator=g).tolist()
    check_fork(R, 1, bs, lengths, NB, parent, 16, 1)
    check_resize(R, 1, bs, lengths, NB, delta, 16, 1)
    check_compact(R, 1, bs, lengths, NB, 16, 1)


def test_a_row_of_many_pages():
    MB = 1 << 18
    check_resize(2, MB, 1, [1000, 5], 600_000, [MB - 1000, 100_000], 16, 1)
    check_resize(2, MB, 1, [MB, 5], 600_000, [-MB, MB - 5], 16, 1)
    check_fork(2, MB, 4, [4 * MB - 1, 77], 600_000, [0, 0, 1], 16, 1)
