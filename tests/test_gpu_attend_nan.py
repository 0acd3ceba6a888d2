"""Attention of queries and over keys that are not finite, where rows see them: the rows are NaN, the others are not
touched by it, and a call of nothing else takes as long as any."""
import math

import pytest
import torch

from tests import forward_support as F
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu

HEADS = [(64, 2, 4, (1, 1)), (64, 2, 4, (30, 33)), (128, 2, 4, (1, 1)), (128, 2, 4, (40, 3)), (576, 1, 4, (1, 1)),
         (576, 1, 20, (1, 1)), (576, 1, 4, (40, 9))]


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d,hk,hq,q", HEADS)
@pytest.mark.parametrize("kv", [(150, 70), (1500, 300)])
def test_queries_that_are_not_finite(d, hk, hq, q, kv, bad):
    c = Case(hq=hq, hk=hk, d=d, kv=kv, q=q, page=16)
    c.q[::3, ::2, 5] = bad
    c.host[0][c.layer, :, 5::d] = 1.0  # so that an infinite query's scores are all of one sign
    c.upload()
    got = c.run()
    torch.cuda.synchronize()
    out, lse = got
    w, wl, tol, tol_l = c.want()
    hit = torch.zeros(wl.shape, dtype=torch.bool)
    hit[::3, ::2] = True
    if bad == -math.inf:  # every visible score is -infinity
        assert out[hit.cuda()].eq(0).all() and lse[hit.cuda()].eq(-math.inf).all()
    else:
        assert out[hit.cuda()].isnan().all() and lse[hit.cuda()].isnan().all()
    F.close(out.cpu()[~hit], w[~hit], tol[~hit], "out")
    F.close(lse.cpu()[~hit], wl[~hit], tol_l[~hit], "lse")
    c.pool.sync()
    c.close()


@pytest.mark.parametrize("kw", [dict(), dict(window=60, sinks=2)])
@pytest.mark.parametrize("d,hk,hq,q", HEADS)
@pytest.mark.parametrize("kv", [(150, 70), (1500, 300)])
def test_keys_that_are_nan(d, hk, hq, q, kv, kw):
    """A NaN key in front of the new tokens and one among them: rows that see one are NaN, and rows of the same tile
    that do not are as without it."""
    c = Case(hq=hq, hk=hk, d=d, kv=kv, q=q, page=16)
    c.host[0][c.layer, F.slots_of(c.table[0], kv[0], c.entry)[kv[0] - max(q[0] // 2, 1)], 5] = math.nan
    c.host[0][c.layer, F.slots_of(c.table[1], kv[1], c.entry)[kv[1] - 61], 5] = math.nan
    c.upload()
    got = c.run(**kw)
    torch.cuda.synchronize()
    out, lse = got
    for s in range(2):
        bad = kv[0] - max(q[0] // 2, 1) if s == 0 else kv[1] - 61
        for r in range(int(c.q_start[s]), int(c.q_start[s + 1])):
            p = kv[s] - int(c.q_start[s + 1]) + r
            sees = bool(F.seen(p, torch.tensor([bad]), True, kw.get("window", 0), kw.get("sinks", 0)))
            heads = slice(0, hq // hk)  # of KV head 0, which has the NaN
            assert out[r, heads].isnan().all() == sees and out[r, heads].isnan().any() == sees, (s, r)
            assert lse[r, heads].isnan().all() == sees and lse[r, heads].isnan().any() == sees, (s, r)
    w, wl, tol, tol_l = c.want(**kw)
    rest = ~lse.isnan().cpu()
    assert rest.any() or q == (1, 1)
    F.close(out.cpu()[rest], w[rest], tol[rest], "out")
    F.close(lse.cpu()[rest], wl[rest], tol_l[rest], "lse")
    c.pool.sync()
    c.close()


@pytest.mark.parametrize("d,hq,hk,m", [(128, 32, 8, 512), (64, 32, 8, 512), (576, 16, 1, 256), (576, 16, 1, 1)])
def test_nan_queries_take_no_longer(d, hq, hk, m):
    n, page = 4096, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    dev = [torch.randn((1, n, hk * d), generator=g, device="cuda").bfloat16() for _ in range(1 if d == 576 else 2)]
    pool = F.pool_of(dev, page, stream=torch.cuda.current_stream())
    table, kv = torch.arange(n // page).cuda()[None], torch.tensor([n]).cuda()
    start = torch.tensor([0, m]).cuda()

    def time(q):
        def run():
            return pool.attend(0, q, table, kv, kv_heads=hk, q_start=start, max_q=m, max_kv=n, return_lse=True,
                               value_dim=512 if d == 576 else d)
        run()
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            out, lse = run()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best, out, lse

    q = torch.randn((m, hq, d), generator=g, device="cuda").bfloat16()
    plain, out, lse = time(q)
    assert out.isfinite().all()
    slow, out, lse = time(torch.full_like(q, math.nan))
    assert out.isnan().all() and lse.isnan().all()
    # rows done one after the other took 6 (decoding) to 110 times as long; 4 leaves room for clocks and the machine
    assert slow < 4 * plain + 0.05, (plain, slow)
    pool.close()
