"""What the forward-pass kernels report of bad lists, and hc_pool_sync beside them."""
import re

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int64).cuda()


@pytest.fixture
def pool():
    dev = [torch.zeros((1, 64, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p = F.pool_of(dev, 16)
    p.keep = dev
    yield p
    torch.cuda.synchronize()
    p.close()


def reports(pool):
    """(code, position) of everything a sync reports, until it reports nothing."""
    out = []
    for _ in range(4):
        try:
            pool.sync()
            return out
        except B.HcError as e:
            assert e.code == B.HC_ERR_DEVICE
            out.append(tuple(int(x) for x in re.search(r"code (\d+):.*position (\d+)", str(e)).groups()))
    raise AssertionError(out)


def test_no_report_is_lost_beside_a_sync(pool):
    """Bad calls of both kinds on a stream that the pool does not know, syncs at any time among them:
    every round's reports arrive, none twice, each with its position."""
    s = torch.cuda.Stream()
    src, dst = ints([1] * 40 + [9]), ints([2] * 40 + [3])
    dst[:40] = 1                                     # page 1 onto itself, then a page that is not there
    table, lens = torch.zeros((30, 1), dtype=torch.int64, device="cuda"), ints([0] * 29 + [99])
    torch.cuda.synchronize()
    for _ in range(50):
        pool.copy_pages(src, dst, stream=s)          # index, position 40
        got = reports(pool)
        pool.free_pages(table, lens, stream=s)       # lengths, position 29
        got += reports(pool)
        s.synchronize()
        got += reports(pool)
        assert sum(c & 1 for c, _ in got) == 1 and sum(c >> 2 & 1 for c, _ in got) == 1, got
        assert all(p == (29 if c & 4 else 40) for c, p in got), got
    assert reports(pool) == []


def test_transfers_and_operators_in_one_report(pool):
    staging = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    pool.layer_pack(0, ints([0, 1, 2, 64]), staging)         # position 3, on the copy stream
    pool.copy_pages(ints([1, 7]), ints([1, 2]))              # position 1
    torch.cuda.synchronize()
    assert reports(pool) == [(1, 1)]
    pool.layer_pack(0, ints([0, 1, 2, 64]), staging)
    pool.free_pages(torch.zeros((9, 1), dtype=torch.int64, device="cuda"), ints([0] * 8 + [-1]))
    torch.cuda.synchronize()
    assert reports(pool) == [(5, 3)]
    pool.layer_pack(0, ints([0, 64]), staging)
    torch.cuda.synchronize()
    assert reports(pool) == [(1, 1)]
