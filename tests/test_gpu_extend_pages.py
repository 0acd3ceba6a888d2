"""Pages, slots and positions of a batch's new tokens, against a plain walk over its rows."""
import ctypes

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu


def pool_of(pages, page):
    dev = [torch.zeros((1, pages * page, 16), dtype=torch.uint8, device="cuda")]
    return F.pool_of(dev, page)


def walk(table, lens, added, free, room, page, pages, first=0):
    """(table, kv_len, q_start, slots, positions, used), and the rows that are reported."""
    table = [list(r) for r in table]
    most = len(table[0]) * page if table else 0
    kv, start, slots, pos, used, bad = [], [0], [-1] * room, [0] * room, 0, set()
    for s, (n, m) in enumerate(zip(lens, added)):
        if n < 0 or n > most or m < 0 or m > room or n + m > most:
            bad.add(s)
            m = 0
        held = -(-n // page) if n >= 0 else 0
        for j in range(m):
            t, e = start[-1] + j, (n + j) // page
            if t >= room:
                bad.add(s)
                continue
            if e >= held:
                k = first + used + e - held
                ident = free[k] if 0 <= first and k < len(free) else -1
                if not 0 <= ident < pages:
                    ident = -1
                if (n + j) % page == 0:
                    table[s][e] = ident
            else:
                ident = table[s][e]
            ok = 0 <= ident < pages
            if not ok:
                bad.add(s)
            slots[t], pos[t] = (ident * page + (n + j) % page if ok else -1), n + j
        if m:
            used += -(-(n + m) // page) - held
        kv.append(n + m)
        start.append(start[-1] + m)
    return (table, kv, start, slots, pos, [used]), bad


def make(lens, page, width, spare, seed):
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) if 0 <= n <= width * page else 0 for n in lens]
    pages = sum(held) + spare
    place = torch.randperm(pages, generator=g).tolist()
    table, at = [], 0
    for h in held:
        table.append(place[at:at + h] + [-7] * (width - h))
        at += h
    return table, place[at:], pages


def run(lens, added, *, page=16, width=8, room=None, spare=64, seed=0, free=None, first=None, table=None):
    made, free_list, pages = make(lens, page, width, spare, seed)
    table = made if table is None else table
    free = free_list if free is None else free
    room = max(0, sum(added)) if room is None else room
    pool = pool_of(pages, page)
    dev = torch.tensor(table, dtype=torch.int64).reshape(len(lens), width).cuda()
    l, a, f = (torch.tensor(x, dtype=torch.int64).cuda() for x in (lens, added, free))
    first_dev = None if first is None else torch.tensor([first]).cuda()
    got = pool.extend_pages(dev, l, a, f, tokens=room, first_free=first_dev)
    want, bad = walk(table, lens, added, free, room, page, pages, first or 0)
    if bad:
        with pytest.raises(B.HcError) as e:
            pool.sync()
        assert e.value.code == B.HC_ERR_DEVICE and str(min(bad)) in str(e.value)
    pool.sync()
    for name, x, y in zip(("table", "kv_len", "q_start", "slots", "positions", "used"), (dev,) + tuple(got), want):
        assert x.cpu().tolist() == y, name
    pool.close()


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("lens,added", [
    ([0], [1]), ([0], [0]), ([15], [1]), ([16], [1]), ([17], [30]), ([5, 0, 16, 31], [1, 1, 1, 1]),
    ([3, 7, 0, 16, 2], [0, 20, 0, 5, 0]), ([0, 0, 0], [0, 0, 0]), ([1, 2, 3, 4], [40, 0, 1, 17])])
def test_small(lens, added, page):
    run(lens, added, page=page, width=-(-64 // page), spare=200)
    run(lens, added, page=page, width=-(-64 // page), spare=200, room=sum(added) + 7, seed=1)


@pytest.mark.parametrize("rows", [63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 3000])
def test_many_rows(rows):
    """More rows than a workgroup has threads, more tokens than it takes; rows that add nothing among them."""
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, 100, (rows,), generator=g).tolist()
    added = [0 if x < 3 else x - 2 for x in torch.randint(0, 9, (rows,), generator=g).tolist()]
    run(lens, added, page=8, width=16, spare=3 * rows, room=sum(added) + 100)


def test_prompts_beside_decoding_rows():
    lens = [500] * 20 + [0, 64, 0, 1000] + [31] * 20
    added = [1] * 20 + [2500, 1100, 3, 700] + [1] * 20
    run(lens, added, page=64, width=60, spare=120, room=5000)


def test_first_free():
    run([5, 16], [20, 20], first=3)
    run([5, 16], [20, 20], first=0)


def test_too_few_pages():
    run([5, 16, 0], [20, 20, 5], free=[3, 1])
    run([5, 16, 0], [20, 20, 5], free=[])
    run([5, 16, 0], [20, 20, 5], first=62)
    run([5, 16, 0], [20, 20, 5], first=-1)
    run([5, 16, 0], [20, 20, 5], first=1 << 62)


def test_pages_outside_the_pool():
    made, free, pages = make([5, 16, 20], 16, 8, 64, 0)
    run([5, 16, 20], [20, 20, 5], free=[free[0], 10 ** 9, -5] + free[3:])
    made[2][1] = pages
    made[0][0] = -1
    run([5, 16, 20], [20, 20, 5], table=made)


@pytest.mark.parametrize("lens,added", [([5, -1, 3], [1, 1, 1]), ([5, 129, 3], [1, 0, 1]), ([5, 128, 3], [1, 1, 1]),
                                        ([5, 10, 3], [1, -1, 1]), ([5, 10, 3], [1, 1 << 62, 1]),
                                        ([5, 1 << 62, 3], [1, 1 << 62, 1]), ([127, 128, 0], [1, 0, 128])])
def test_lengths_out_of_bounds(lens, added):
    run(lens, added, room=140)


def test_too_little_room():
    run([5, 16, 20, 0], [10, 10, 10, 0], room=15)
    run([5, 16, 20, 0], [10, 10, 10, 0], room=10)
    run([5, 16], [1, 1], room=0)


def test_strided_table_and_empty_calls():
    pool = pool_of(16, 16)
    wide = torch.full((3, 11), -7, dtype=torch.int64, device="cuda")
    lens, added = torch.tensor([0, 0, 0]).cuda(), torch.tensor([17, 0, 16]).cuda()
    free = torch.arange(16, device="cuda")
    got = pool.extend_pages(wide[:, 2:6], lens, added, free, tokens=40)
    want = torch.full((3, 11), -7)
    want[0, 2:4], want[2, 2] = torch.tensor([0, 1]), 2
    assert torch.equal(wide.cpu(), want) and got[4].item() == 3
    empty = torch.zeros((0, 4), dtype=torch.int64, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    kv, start, slots, pos, used = pool.extend_pages(empty, none, none, none, tokens=5)
    assert kv.numel() == 0 and start.tolist() == [0] and slots.tolist() == [-1] * 5 and pos.tolist() == [0] * 5
    assert used.item() == 0
    pool.sync()
    pool.close()


def test_captured_steps():
    """A decoding step's lists in one graph: lengths and the free list's start move on the device."""
    pool = pool_of(64, 4)
    g = torch.Generator().manual_seed(1)
    free = torch.randperm(64, generator=g)
    table = torch.full((3, 8), -1, dtype=torch.int64)
    table[0, 0], table[1, :2] = free[0], free[1:3]
    lens0 = [3, 8, 0]
    dev, lens, first = table.cuda(), torch.tensor(lens0).cuda(), torch.tensor([3]).cuda()
    added, pages = torch.tensor([1, 1, 1]).cuda(), free.cuda()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        kv, start, slots, pos, used = pool.extend_pages(dev, lens, added, pages, tokens=4, first_free=first)
        lens.copy_(kv)
        first += used
    want_table, want_lens, at = table.tolist(), lens0, 3
    for step in range(9):
        graph.replay()
        torch.cuda.synchronize()
        (want_table, want_lens, w_start, w_slots, w_pos, w_used), bad = walk(want_table, want_lens, [1, 1, 1],
                                                                            free.tolist(), 4, 4, 64, at)
        at += w_used[0]
        assert not bad
        assert dev.tolist() == want_table and lens.tolist() == want_lens and slots.tolist() == w_slots
        assert start.tolist() == w_start and pos.tolist() == w_pos and first.item() == at
    pool.sync()
    del graph
    pool.close()


def test_refusals():
    pool = pool_of(16, 16)
    ints = torch.zeros(200, dtype=torch.int64, device="cuda")
    good = dict(table=0, table_rows=2, table_width=4, table_stride=4, lens=10, added=14, free_pages=20, n_free=8,
                first_free=30, kv_len=40, q_start=50, slots=60, positions=80, room=10, used=100)
    where = ("table", "lens", "added", "free_pages", "first_free", "kv_len", "q_start", "slots", "positions", "used")

    def call(**kw):
        d = B.hc_extend_desc()
        for k, v in dict(good, **kw).items():
            setattr(d, k, ints[v:].data_ptr() if k in where and v is not None else v)
        return B.lib.hc_extend_pages(pool.handle, ctypes.byref(d), None)

    assert call() == B.HC_OK
    assert call(first_free=None) == B.HC_OK
    for kw in [dict(table_rows=-1), dict(table_stride=3), dict(n_free=-1), dict(room=-1), dict(room=1 << 31), dict(table=None),
               dict(lens=None), dict(slots=None), dict(used=None), dict(kv_len=1), dict(q_start=41), dict(slots=45),
               dict(positions=61), dict(used=65), dict(kv_len=10), dict(slots=6), dict(table=14), dict(used=30),
               dict(q_start=21)]:
        assert call(**kw) == B.HC_ERR_INVALID, kw
    # written lists stay in device memory
    host = torch.zeros(8, dtype=torch.int64).pin_memory()
    d = B.hc_extend_desc()
    for k, v in good.items():
        setattr(d, k, ints[v:].data_ptr() if k in where else v)
    d.kv_len = host.data_ptr()
    assert B.lib.hc_extend_pages(pool.handle, ctypes.byref(d), None) == B.HC_ERR_INVALID
    d.kv_len, d.lens = ints[40:].data_ptr(), host.data_ptr()  # read ones may be pinned
    assert B.lib.hc_extend_pages(pool.handle, ctypes.byref(d), None) == B.HC_OK
    table = torch.zeros((2, 4), dtype=torch.int64, device="cuda")
    two = torch.zeros(2, dtype=torch.int64, device="cuda")
    for args, kw in [((table, two[:1], two, two), dict(tokens=4)), ((table, two, two, two), dict(tokens=-1)),
                     ((table, two, two, two), dict(tokens=4, first_free=two))]:
        with pytest.raises(ValueError):
            pool.extend_pages(*args, **kw)
    torch.cuda.synchronize()
    pool.sync()
    pool.close()
