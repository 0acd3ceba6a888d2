"""Page tables with entries and lengths that name nothing, in every place of a row."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu

PAGE, PAGES = 16, 20


def ints(x):
    return torch.tensor(x, dtype=torch.int64).cuda()


@pytest.fixture
def pool():
    g = torch.Generator().manual_seed(2)
    dev = [torch.randint(0, 256, (2, PAGES * PAGE, 64), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    p = F.pool_of(dev, PAGE)
    p.keep, p.before = dev, [t.clone() for t in dev]
    yield p
    torch.cuda.synchronize()
    p.close()


def reported(pool, words):
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match=words):
        pool.sync()
    pool.sync()


@pytest.mark.parametrize("bad", [PAGES, -1, -(1 << 60), 1 << 60])
@pytest.mark.parametrize("rest", [0, 5])
def test_fork_of_a_row_with_a_bad_full_page(pool, bad, rest):
    """A parent of whole pages, and one with a partly filled last page: the child never gets the entry."""
    table = ints([[3, 4, 5, 6], [7, bad, 9, 10]])
    lens = ints([4 * PAGE, 3 * PAGE + rest])
    out = torch.full((3, 4), 77, dtype=torch.int64, device="cuda")
    used = pool.fork_pages(table, lens, ints([0, 1, 0]), ints([15, 16]), out)
    reported(pool, "index out of range; first flagged list position 1")
    assert out.tolist() == [[3, 4, 5, 6], [7, -1, 9, 15 if rest else -1], [3, 4, 5, 6]]
    assert used.item() == (1 if rest else 0)
    want = [t.clone() for t in pool.before]
    for t in want:
        t[:, 15 * PAGE:15 * PAGE + rest] = t[:, 10 * PAGE:10 * PAGE + rest]
    assert all(torch.equal(a, b) for a, b in zip(pool.keep, want))


def test_entries_behind_a_length_are_not_read(pool):
    table = ints([[3, 1 << 60], [4, -5]])
    out = torch.full((2, 2), 77, dtype=torch.int64, device="cuda")
    pool.fork_pages(table, ints([PAGE, 0]), ints([0, 1]), ints([15]), out)
    pool.sync()
    assert out.tolist() == [[3, -1], [-1, -1]]


@pytest.mark.parametrize("pages", [20, 131073])
def test_lengths_of_a_table_without_entries(pages):
    """Rows of no entries: a length above 0 is out of bounds like any other, on both sides of what one
    workgroup scans."""
    dev = [torch.zeros((1, pages, 16), dtype=torch.uint8, device="cuda")]
    pool = F.pool_of(dev, 1)
    empty = torch.empty((300, 0), dtype=torch.int64, device="cuda")
    lens = torch.zeros(300, dtype=torch.int64)
    free, n = pool.free_pages(empty, lens.cuda())
    assert n.item() == pages and torch.equal(free.cpu(), torch.arange(pages))
    assert pool.compact_pages(empty, lens.cuda(), empty).item() == 0
    pool.sync()
    lens[280:] = 1
    for call in (lambda: pool.free_pages(empty, lens.cuda())[1], lambda: pool.compact_pages(empty, lens.cuda(), empty)):
        assert call().item() in (0, pages)
        reported(pool, "lengths out of bounds; first flagged list position 280")
    pool.close()
