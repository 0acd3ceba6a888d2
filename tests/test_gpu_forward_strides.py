"""Strides of dimensions of one element, which torch may report as anything."""
import pytest
import torch

from tests import forward_support as F

pytestmark = pytest.mark.gpu

DT = torch.bfloat16


def odd(t, dim):
    """The same tensor with an odd stride in a dimension of one element."""
    stride = list(t.stride())
    assert t.shape[dim] == 1
    stride[dim] = 3
    return t.as_strided(t.shape, stride)


def normal(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float64).to(DT).cuda()


@pytest.mark.parametrize("n,hq,hk", [(1, 4, 2), (5, 1, 1), (1, 1, 1)])
def test_single_tokens_and_heads(n, hq, hk):
    g = torch.Generator().manual_seed(n + hq)
    dev = [torch.zeros((1, 64, hk * 64), dtype=DT, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    q, k, v = normal(g, n, hq, 64), normal(g, n, hk, 64), normal(g, n, hk, 64)
    qs, ks, vs = q.clone(), k.clone(), v.clone()
    for dim, count in ((0, n), (1, hk)):
        if count == 1:
            ks, vs = odd(ks, dim), odd(vs, dim)
    for dim, count in ((0, n), (1, hq)):
        if count == 1:
            qs = odd(qs, dim)
    out = torch.empty_strided(qs.shape, qs.stride(), dtype=DT, device="cuda")
    pool.store_tokens(0, torch.arange(n).cuda(), ks, vs, q=qs, q_out=out)
    torch.cuda.synchronize()
    assert torch.equal(F.bits(out), F.bits(q))
    assert torch.equal(F.bits(dev[0][0, :n].view(n, hk, 64)), F.bits(k))
    assert torch.equal(F.bits(dev[1][0, :n].view(n, hk, 64)), F.bits(v))
    # in place, the same memory under other strides of its single token or head
    pool.store_tokens(0, torch.arange(n).cuda(), ks, vs, q=q.clone(), q_out=qs)
    same = q.clone()
    view = same
    for dim, count in ((0, n), (1, hq)):
        if count == 1:
            view = odd(view, dim)
    pool.store_tokens(0, torch.arange(n).cuda(), ks, vs, q=same, q_out=view)
    got, lse = pool.attend(0, qs, torch.arange(4).cuda()[None], torch.tensor([n]).cuda(), kv_heads=hk,
                           q_start=torch.tensor([0, n]).cuda(), out=out, return_lse=True)
    torch.cuda.synchronize()
    w, wl, tol, tol_l = F.attend(q.cpu(), k.flatten(1).cpu(), v.flatten(1).cpu(), torch.arange(n)[None], [n], [0, n],
                                 kv_heads=hk, entry=1)
    F.close(out, w, tol, "out")
    F.close(lse, wl, tol_l, "lse")
    pool.sync()
    pool.close()


def test_a_single_row_table_in_place_under_another_stride():
    dev = [torch.arange(64, dtype=torch.float32).view(1, 64, 1).expand(1, 64, 4).contiguous().cuda()]
    pool = F.pool_of(dev, 16)
    table = torch.tensor([[3, 1]]).cuda()
    assert pool.compact_pages(table, torch.tensor([20]).cuda(), table.as_strided((1, 2), (9, 1))).item() == 2
    torch.cuda.synchronize()
    pool.sync()
    assert table.tolist() == [[0, 1]] and dev[0][0, :16, 0].tolist() == [float(48 + i) for i in range(16)]
    pool.close()
