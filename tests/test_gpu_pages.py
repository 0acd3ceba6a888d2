"""Page tables over the device pool: copies, forks, free lists and compaction, byte for byte
against a plain implementation on lists."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu


class Pages:
    """A pool of K and V rows and, if asked, one block per page, filled with random bytes."""

    def __init__(self, page=16, pages=40, layers=3, rows=(256, 96), block=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.pages = page, pages
        self.host = [torch.randint(0, 256, (layers, pages * page, e), generator=g, dtype=torch.uint8) for e in rows]
        if block:
            self.host.append(torch.randint(0, 256, (layers, pages, block), generator=g, dtype=torch.uint8))
        self.dev = [t.cuda() for t in self.host]
        self.block = len(rows) if block else None
        self.pool = F.pool_of(self.dev, page, blocks=[self.block] if block else ())
        self.g = g

    def copied(self, moves):
        """The pool after (from, to, rows) moves whose sources are read before any write."""
        out = [t.clone() for t in self.host]
        for a, b, rows in moves:
            for i, t in enumerate(out):
                if i == self.block:
                    t[:, b] = self.host[i][:, a]
                else:
                    p = self.page
                    t[:, b * p:b * p + rows] = self.host[i][:, a * p:a * p + rows]
        return out

    def check(self, moves):
        torch.cuda.synchronize()
        for i, (got, want) in enumerate(zip(self.dev, self.copied(moves))):
            assert torch.equal(got.cpu(), want), f"sub {i}"

    def table(self, lens, width=None, shared=0):
        """Rows of random distinct pages, the first `shared` entries the same in every row."""
        n = [-(-x // self.page) for x in lens]
        width = max(n + [1]) if width is None else width
        place = torch.randperm(self.pages, generator=self.g).tolist()
        head = [place.pop() for _ in range(shared)]
        t = torch.full((len(lens), width), -7, dtype=torch.int64)
        for s, k in enumerate(n):
            for j in range(k):
                t[s, j] = head[j] if j < shared else place.pop()
        return t, place

    def close(self):
        self.pool.close()


def ints(x):
    return torch.tensor(x, dtype=torch.int64).cuda()


@pytest.mark.parametrize("kw", [dict(), dict(page=1, pages=200, rows=(16,)), dict(block=8448, rows=(1152,), page=64, pages=12),
                                dict(page=64, pages=9, rows=(2048, 2048), layers=5), dict(page=7, rows=(48,), layers=1)])
def test_copy(kw):
    p = Pages(**kw)
    order = torch.randperm(p.pages, generator=p.g).tolist()
    src = order[:4] + [order[0], order[8], order[2]]       # a source may repeat
    dst = [order[4], order[5], order[2], order[6], order[7], order[8], order[3]]
    src[2], src[6] = order[0], order[1]                    # targets are nobody's source, or their own
    dst[2], dst[6] = order[9 % p.pages] if p.pages > 9 else order[4], order[10 % p.pages] if p.pages > 10 else order[5]
    pairs = {b: a for a, b in zip(src, dst)}
    pairs = {b: a for b, a in pairs.items() if a == b or b not in pairs.values()}
    p.pool.copy_pages(ints(list(pairs.values())), ints(list(pairs)))
    p.pool.copy_pages(ints([]), ints([]))
    p.pool.sync()
    p.check([(a, b, p.page) for b, a in pairs.items()])
    p.close()


def test_copy_reports_bad_pages():
    p = Pages()
    p.pool.copy_pages(ints([1, 40, 3, -1, 1 << 60]), ints([2, 5, 40, 6, 7]))
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="first flagged list position 1"):
        p.pool.sync()
    p.check([(1, 2, 16)])
    p.close()


def forked(p, table, lens, parents, free):
    rows, moves, used = [], [], 0
    for r in parents:
        full, rest = divmod(lens[r], p.page)
        row = table[r][:full].tolist()
        if rest:
            if used < len(free):
                moves.append((int(table[r][full]), free[used], rest))
                row.append(free[used])
            else:
                row.append(-1)
            used += 1
        rows.append(row + [-1] * (table.shape[1] - len(row)))
    return torch.tensor(rows), used, moves


@pytest.mark.parametrize("kw", [dict(), dict(page=1, pages=300, rows=(16,)),
                                dict(block=8448, rows=(1152,), page=64, pages=40, layers=2)])
def test_fork(kw):
    p = Pages(**kw)
    P = p.page
    lens = [3 * P + P // 2, P, 0, 2 * P + 1, 1, 4 * P - 1 if P > 1 else 4]
    table, free = p.table(lens, width=6)
    parents = [0, 3, 0, 1, 2, 5, 4, 0, 3]
    out = torch.full((len(parents), 6), 99, dtype=torch.int64, device="cuda")
    used = p.pool.fork_pages(table.cuda(), ints(lens), ints(parents), ints(free), out)
    p.pool.sync()
    want, n, moves = forked(p, table, lens, parents, free)
    assert torch.equal(out.cpu(), want) and used.tolist() == [n]
    p.check(moves)
    p.close()


def test_fork_many_children_of_a_strided_table():
    """More children than one step of the numbering takes, into rows of a wider table."""
    p = Pages(page=4, pages=3000, rows=(16,), layers=2)
    lens = [7, 8, 9]
    table, free = p.table(lens, width=3)
    wide = torch.full((3, 9), -5, dtype=torch.int64, device="cuda")
    wide[:, :3] = table.cuda()
    parents = torch.randint(0, 3, (2500,), generator=p.g).tolist()
    big = torch.full((2500, 8), 77, dtype=torch.int64, device="cuda")
    used = p.pool.fork_pages(wide[:, :3], ints(lens), ints(parents), ints(free), big[:, 2:5])
    p.pool.sync()
    want, n, moves = forked(p, table, lens, parents, free)
    assert torch.equal(big[:, 2:5].cpu(), want) and used.item() == n
    assert big[:, :2].eq(77).all() and big[:, 5:].eq(77).all()
    p.check(moves)
    p.close()


def test_fork_reports_what_it_cannot_do():
    p = Pages()
    lens = [20, 33, 16]
    table, free = p.table(lens, width=3)
    # too few free pages
    out = torch.zeros((3, 3), dtype=torch.int64, device="cuda")
    used = p.pool.fork_pages(table.cuda(), ints(lens), ints([0, 1, 0]), ints(free[:2]), out)
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="first flagged list position 2"):
        p.pool.sync()
    want, n, moves = forked(p, table, lens, [0, 1, 0], free[:2])
    assert torch.equal(out.cpu(), want) and used.item() == 3
    p.check(moves)
    # bad parents, lengths, entries and free pages: nothing else moves
    before = [t.clone() for t in p.dev]
    bad = table.clone()
    bad[0, 1] = 1 << 40
    out.zero_()
    p.pool.fork_pages(bad.cuda(), ints([20, -1, 16]), ints([0, 1, 3]), ints(free), out)
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="code 5"):
        p.pool.sync()
    assert out.tolist() == [[int(table[0, 0]), free[0], -1], [-1] * 3, [-1] * 3]
    p.pool.fork_pages(table.cuda(), ints(lens), ints([0]), ints([40]), out[:1])
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="out of range"):
        p.pool.sync()
    assert out[0].tolist() == [int(table[0, 0]), -1, -1]
    assert all(torch.equal(a, b) for a, b in zip(before, p.dev))
    p.pool.fork_pages(table.cuda(), ints(lens), ints([]), ints([]), out[:0])  # no child
    p.pool.sync()
    p.close()


def packed(p, table, lens):
    n = [-(-x // p.page) if 0 <= x <= table.shape[1] * p.page else 0 for x in lens]
    live = sorted({int(x) for s, k in enumerate(n) for x in table[s, :k] if 0 <= x < p.pages})
    count = len(live)
    holes = [x for x in range(count) if x not in live]
    to = dict(zip([x for x in live if x >= count], holes))
    out = table.clone()
    for s, k in enumerate(n):
        for j in range(k):
            out[s, j] = to.get(int(table[s, j]), int(table[s, j]))
    return out, count, [(a, b, p.page) for a, b in to.items()], [x for x in range(p.pages) if x not in live]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(page=1, pages=2500, rows=(16,), layers=1), dict(pages=1100, rows=(16, 32)),
                                dict(block=8448, rows=(1152,), page=64, pages=40, layers=2)])
def test_compact_and_free_list(kw, in_place):
    p = Pages(**kw)
    P = p.page
    lens = [5 * P, 0, 4 * P + 1 if P > 1 else 5, 3 * P, 2 * P]
    table, _ = p.table(lens, width=7, shared=2)
    on, ln = table.cuda(), ints(lens)
    want, count, moves, free = packed(p, table, lens)
    pages, n = p.pool.free_pages(on, ln)
    assert n.tolist() == [len(free)] and pages[:len(free)].tolist() == free
    out = on if in_place else torch.full_like(on, 55)
    live = p.pool.compact_pages(on, ln, out)
    p.pool.sync()
    assert live.tolist() == [count] and torch.equal(out.cpu(), want)
    p.check(moves)
    # once packed, nothing moves any more
    again = p.pool.compact_pages(out, ln, torch.empty_like(out))
    p.check(moves)
    pages, n = p.pool.free_pages(out, ln)
    assert again.item() == count and pages[:n.item()].tolist() == list(range(count, p.pages))
    p.close()


@pytest.mark.parametrize("pages,rows,width", [(140001, 3, 200), (3000, 400, 100), (131072, 2, 33), (33, 8, 5)])
def test_compact_large_pools_and_tables(pages, rows, width):
    """Pools and tables on both sides of what one workgroup scans, the last page named."""
    p = Pages(page=1, pages=pages, rows=(16,), layers=1)
    table = torch.randint(0, pages, (rows, width), generator=p.g)
    table[0, 0] = pages - 1
    lens = torch.randint(0, width + 1, (rows,), generator=p.g)
    lens[0] = width
    live = torch.zeros(pages, dtype=torch.bool)
    live[torch.cat([table[s, :n] for s, n in enumerate(lens)])] = True
    count = int(live.sum())
    ids = torch.arange(pages)
    source, target = ids[live & (ids >= count)], ids[~live & (ids < count)]
    moved = ids.clone()
    moved[source] = target
    want = torch.where(torch.arange(width)[None] < lens[:, None], moved[table], table)
    free, n = p.pool.free_pages(table.cuda(), lens.cuda())
    assert n.item() == pages - count and torch.equal(free[:n.item()].cpu(), ids[~live])
    out = torch.empty_like(table).cuda()
    assert p.pool.compact_pages(table.cuda(), lens.cuda(), out).item() == count
    p.pool.sync()
    assert torch.equal(out.cpu(), want)
    after = p.host[0].clone()
    after[:, target] = p.host[0][:, source]
    assert torch.equal(p.dev[0].cpu(), after)
    p.close()


def test_compact_full_empty_and_bad_tables():
    p = Pages(pages=8)
    table = torch.randperm(8, generator=p.g).view(2, 4)
    out = torch.empty_like(table).cuda()
    assert p.pool.compact_pages(table.cuda(), ints([64, 64]), out).item() == 8  # every page live
    assert torch.equal(out.cpu(), table)
    assert p.pool.free_pages(table.cuda(), ints([64, 64]))[1].item() == 0
    assert p.pool.compact_pages(table.cuda(), ints([0, 0]), out).item() == 0    # none
    assert torch.equal(out.cpu(), table)
    empty = torch.empty((0, 4), dtype=torch.int64, device="cuda")
    assert p.pool.compact_pages(empty, ints([]), empty).item() == 0
    assert p.pool.free_pages(empty, ints([]))[1].item() == 8
    p.pool.sync()
    p.check([])
    bad = torch.tensor([[7, 9, -3, 2], [6, 1, 0, 3]])
    lens = [50, 1000]
    want, count, moves, _ = packed(p, bad, lens)
    assert p.pool.compact_pages(bad.cuda(), ints(lens), out).item() == count == 2
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="code 5"):
        p.pool.sync()
    assert torch.equal(out.cpu(), want)
    p.check(moves)
    p.close()


def test_refusals():
    p = Pages()
    table, lens = torch.zeros((2, 3), dtype=torch.int64, device="cuda"), ints([1, 1])

    def refuse(call):
        with pytest.raises(B.HcError) as e:
            call()
        assert e.value.code == B.HC_ERR_INVALID, e.value

    refuse(lambda: p.pool.fork_pages(table, lens, ints([0, 1]), ints([5]), table))              # in place
    refuse(lambda: p.pool.compact_pages(table[:, :2], lens, table[:, 1:]))                      # overlaps
    lists = torch.zeros(64, dtype=torch.int64, device="cuda")
    refuse(lambda: p.pool.compact_pages(table, lists[:2], lists[:6].view(2, 3)))                # the lengths
    refuse(lambda: p.pool.fork_pages(table, lens, lists[:1], ints([5]), lists[:3].view(1, 3)))  # the parents
    with pytest.raises(ValueError):
        p.pool.fork_pages(table, lens, ints([0]), ints([5]), torch.zeros((1, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        p.pool.compact_pages(table, ints([1]), table)
    with pytest.raises(TypeError):
        p.pool.free_pages(table.int(), lens)
    with pytest.raises(TypeError):
        p.pool.copy_pages(torch.zeros(1, dtype=torch.int64), ints([1]))
    rc = B.lib.hc_free_pages(p.pool.handle, table.data_ptr(), 2, 3, 3, lens.data_ptr(), table.data_ptr(),
                             lens.data_ptr(), table.data_ptr(), 8, None)                        # small workspace
    assert rc == B.HC_ERR_INVALID
    p.check([])
    p.close()
    odd = [torch.zeros((1, 50, 64), dtype=torch.uint8, device="cuda")]
    pool = F.pool_of(odd, 16)                                                                    # 50 slots: no whole pages
    with pytest.raises(B.HcError):
        pool.copy_pages(ints([0]), ints([1]))
    pool.close()


def test_captured_compaction_replays():
    """A captured compaction replayed on tables that change, each replay against the plain one."""
    p = Pages(pages=64)
    on, ln = torch.zeros((4, 5), dtype=torch.int64, device="cuda"), ints([0, 0, 0, 0])
    out = torch.zeros_like(on)
    p.pool.compact_pages(on, ln, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        count = p.pool.compact_pages(on, ln, out)
        pages, n_free = p.pool.free_pages(out, ln)
    for lens in ([80, 17, 0, 33], [1, 2, 3, 64], [80, 80, 80, 80]):
        table, _ = p.table(lens, width=5)
        on.copy_(table)
        ln.copy_(torch.tensor(lens))
        graph.replay()
        torch.cuda.synchronize()
        want, n, moves, _ = packed(p, table, lens)
        assert count.item() == n and torch.equal(out.cpu(), want)
        assert pages[:n_free.item()].tolist() == list(range(n, 64))
        p.check(moves)
        p.host = [t.cpu() for t in p.dev]
    p.pool.sync()
    del graph
    p.close()


def test_pool_destroyed_while_an_operator_runs():
    """Destroying the pool waits for operators on streams other than the copy stream."""
    p = Pages(page=64, pages=512, layers=8, rows=(2048, 2048))
    s = torch.cuda.Stream()
    order = torch.randperm(512, generator=p.g)
    src, dst = order[:256].cuda(), order[256:].cuda()
    torch.cuda.synchronize()
    for _ in range(20):
        p.pool.copy_pages(src, dst, stream=s)
    p.pool.close()
    assert s.query()
    p.check([(int(a), int(b), 64) for a, b in zip(order[:256], order[256:])])
