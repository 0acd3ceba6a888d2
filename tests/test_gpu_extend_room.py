"""Extension of sequences past the room of the call: a table row that named other sequences' pages behind its end does not
come to own them."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests.test_gpu_extend_pages import pool_of, walk

pytestmark = pytest.mark.gpu


def cut(table, lens, added, room, page):
    """(row, entry) of pages that begin with a token past the room."""
    out, start = [], 0
    for s, (n, m) in enumerate(zip(lens, added)):
        out += [(s, (n + j) // page) for j in range(m) if (n + j) % page == 0 and start + j >= room]
        start += m
    return out


# rows, page, room: cut in the first page of a row, inside one, at its end, everything, and nothing; rows behind the cut one, and
# many of them
CASES = [([5, 16, 20, 0], [40, 40, 10, 33], 16, 60), ([5, 16, 20, 0], [40, 40, 10, 33], 16, 40), ([16, 0], [16, 48], 16, 48),
         ([3, 30], [1, 100], 16, 100), ([0], [100], 1, 100), ([0, 0], [60, 60], 1, 100), ([0, 7], [60, 60], 4, 61),
         ([9] * 300, [20] * 300, 8, 3000), ([0] * 1500, [3] * 1500, 2, 2000), ([100, 4], [2500, 2500], 4, 2600)]


@pytest.mark.parametrize("lens,added,page,room", CASES, ids=lambda x: None if isinstance(x, list) else str(x))
def test_pages_without_room(lens, added, page, room):
    g = torch.Generator().manual_seed(len(lens))
    rows = len(lens)
    width = max(-(-(n + 2 * m) // page) for n, m in zip(lens, added)) + 2
    held = [-(-n // page) for n in lens]
    spare = 2 * sum(-(-(n + 2 * m) // page) - h for n, m, h in zip(lens, added, held))
    pages = sum(held) + spare
    place = torch.randperm(pages, generator=g).tolist()
    owned, at = [], 0
    for h in held:
        owned.append(place[at:at + h])
        at += h
    free = place[at:]
    # behind a row's end stand pages of others: of the next rows, and free ones
    others = torch.randint(0, pages, (rows, width), generator=g).tolist()
    table = [o + t[len(o):] for o, t in zip(owned, others)]
    pool = pool_of(pages, page)
    dev = torch.tensor(table).cuda()
    l, a, f = (torch.tensor(x).cuda() for x in (lens, added, free))
    got = pool.extend_pages(dev, l, a, f, tokens=room)
    (want, *lists), bad = walk(table, lens, added, free, room, page, pages)
    lost = cut(table, lens, added, room, page)
    for s, e in lost:
        want[s][e] = -1
    assert bool(bad) == (sum(added) > room)
    if bad:
        with pytest.raises(B.HcError) as err:
            pool.sync()
        assert err.value.code == B.HC_ERR_DEVICE and str(min(bad)) in str(err.value)
    pool.sync()
    for name, x, y in zip(("table", "kv_len", "q_start", "slots", "positions", "used"), (dev,) + tuple(got), [want] + lists):
        assert x.cpu().tolist() == y, name
    # the next step, as a captured one goes on: no token goes to a page that the row was not given
    given = [set(o) for o in owned]
    for s in range(rows):
        given[s] |= {want[s][e] for e in range(held[s], -(-lists[0][s] // page))} - {-1}
    assert sum(map(len, given)) == len(set().union(*given))  # a page has one row
    more = [1] * rows
    first = lists[4][0]
    kv, start, slots, _, _ = pool.extend_pages(dev, got[0], torch.tensor(more).cuda(), f, tokens=rows,
                                               first_free=torch.tensor([first]).cuda())
    after, _ = walk(want, lists[0], more, free, rows, page, pages, first)
    assert dev.cpu().tolist() == after[0] and slots.cpu().tolist() == after[3]
    for s, slot in enumerate(slots.cpu().tolist()):
        fresh = lists[0][s] % page == 0
        assert slot == -1 or slot // page in given[s] or fresh and slot // page in free[first:]
    try:
        pool.sync()
    except B.HcError:
        pass  # (rows that lost pages are reported again)
    pool.close()


def test_entries_outside_the_pool_stay():
    """What names no page of the pool needs no entry in its place."""
    pool = pool_of(20, 4)
    table = torch.tensor([[7, 20, -3, 5], [1, 99, 3, -1]]).cuda()
    lens, added = torch.tensor([2, 4]).cuda(), torch.tensor([12, 10]).cuda()
    pool.extend_pages(table, lens, added, torch.arange(8, 20).cuda(), tokens=12)
    assert table.tolist() == [[7, 8, 9, 10], [1, 99, -1, -1]]
    with pytest.raises(B.HcError):
        pool.sync()
    pool.close()
