"""A step's calls recorded into one graph and replayed on contents that change, against the same calls made eagerly."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,hq,hk,pad,q", [(64, 8, 8, 10000, (1, 1, 1)), (128, 8, 2, 0, (1, 1, 1)), (64, 8, 2, 3, (33, 1, 2)),
                                           (576, 2, 1, 7000, (1, 1, 1)), (576, 70, 1, 0, (3, 1, 1))])
def test_a_step_replayed(d, hq, hk, pad, q):
    """Store, attention (with places for every item's partial result and with fewer), fork and free list."""
    c = Case(hq=hq, hk=hk, d=d, kv=(1500, 70, 900), q=q, page=16, pad_rows=pad).upload()
    n = int(c.q_start[-1])
    rope = B.Rope(rot_dim=64, rot_offset=512 if d == 576 else 0)
    slots = torch.cat([F.slots_of(c.table[s], c.kv[s], 16)[c.kv[s] - c.q_len[s]:] for s in range(3)]).cuda()
    pos = torch.arange(n).cuda()
    q_in, k = torch.empty_like(c.on["q"][:n]), torch.empty((n, hk, d), dtype=c.dt, device="cuda")
    v = None if d == 576 else torch.empty_like(k)
    parents = torch.tensor([2, 0, 1]).cuda()  # a page is left for each
    pages = c.host[0].shape[1] // 16
    free = torch.tensor([p for p in range(pages) if p not in set(c.table.flatten().tolist())]).cuda()
    out = torch.zeros((c.rows, hq, c.dv), dtype=c.dt, device="cuda")
    children = torch.zeros((3, c.table.shape[1]), dtype=torch.int64, device="cuda")

    def step():
        c.pool.store_tokens(1, slots, k, v, q=q_in, q_out=c.on["q"][:n], rope=rope, positions=pos)
        _, lse = c.run(out=out)
        used = c.pool.fork_pages(c.on["table"], c.on["kv_len"], parents, free, children)
        listed, count = c.pool.free_pages(c.on["table"], c.on["kv_len"])
        return [out, lse[:n], children, used, count, listed]

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (q_in, k) + (() if v is None else (v,)):
            t.normal_(generator=g)
        pos.random_(0, 100000, generator=g)
        c.on["kv_len"].copy_(torch.tensor([1500 - 37 * seed, 70, 900 - seed]))

    fill(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        recorded = step()
    for seed in range(4):
        fill(seed)
        eager = [t.clone() for t in step()]
        rows = [t.clone() for t in c.dev]
        n_free = int(eager[4])
        for t in c.dev:
            t[1, slots] = 0
        for t in recorded:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(recorded[:5], eager):
            assert torch.equal(F.bits(a) if a.dtype == c.dt else a, F.bits(b) if b.dtype == c.dt else b)
        assert torch.equal(recorded[5][:n_free], eager[5][:n_free])
        assert all(torch.equal(F.bits(a), F.bits(b)) for a, b in zip(c.dev, rows))
        torch.randn(1000, 1000, device="cuda").sum()
    c.pool.sync()
    del graph
    c.close()
