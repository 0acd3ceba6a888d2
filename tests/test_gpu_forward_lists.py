"""The lists of the forward-pass calls: in pinned host memory, and left out."""
import ctypes

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu


def pinned(x):
    t = torch.empty(x.shape, dtype=torch.int64, pin_memory=True)
    t.copy_(x)
    return t


@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (576, 20, 1)])
@pytest.mark.parametrize("pad", [0, 5])
def test_one_row_a_sequence_without_q_start(d, hq, hk, pad):
    kv = (5, 0, 300, 1500, 64)
    c = Case(hq=hq, hk=hk, d=d, kv=kv, q=(1,) * 5, page=16, pad_rows=pad).upload()
    c.on["q_start"] = None
    out, lse = c.run(max_q=None)
    torch.cuda.synchronize()
    c.pool.sync()
    c.compare(out, lse, c.want())
    # fewer rows than sequences
    with pytest.raises(B.HcError, match="q_rows is below num_seqs"):
        c.pool.attend(1, c.on["q"][:4], c.on["table"], c.on["kv_len"], **c.args)
    c.close()


@pytest.mark.parametrize("d,hq,hk,q", [(128, 4, 2, (1, 1, 1)), (64, 4, 2, (40, 3, 1)), (576, 16, 1, (1, 1, 1))])
def test_attention_over_lists_in_pinned_memory(d, hq, hk, q):
    c = Case(hq=hq, hk=hk, d=d, kv=(900, 33, 64), q=q, page=16).upload()
    start, lens, table = pinned(c.q_start), pinned(c.kv_len), pinned(c.table)
    out = torch.full((c.rows, hq, c.dv), 9.0, dtype=c.dt, device="cuda")
    lse = torch.empty((c.rows, hq), device="cuda")
    a = B.hc_attend_desc(layer=1, dtype=B.HC_BF16, q_heads=hq, kv_heads=hk, head_dim=d, value_dim=c.dv,
                         value_in_key=d == 576, causal=1, entry_tokens=16, scale=d ** -0.5, num_seqs=3, q_rows=c.rows,
                         max_q=max(q), max_kv=900, table_width=table.shape[1], table_stride=table.stride(0))
    a.q, a.out, a.lse, a.q_start, a.kv_len, a.table = (t.data_ptr() for t in (c.on["q"], out, lse, start, lens, table))
    a.q_stride[:], a.out_stride[:] = c.on["q"].stride()[:2], out.stride()[:2]
    need = ctypes.c_int64()
    assert B.lib.hc_attend_workspace_bytes(c.pool.handle, ctypes.byref(a), ctypes.byref(need)) == B.HC_OK
    work = torch.empty(max(need.value, 16), dtype=torch.uint8, device="cuda")
    a.workspace, a.workspace_bytes = work.data_ptr(), need.value
    torch.cuda.synchronize()
    assert B.lib.hc_attend(c.pool.handle, ctypes.byref(a), None) == B.HC_OK, B.lib.hc_last_error()
    torch.cuda.synchronize()
    c.pool.sync()
    c.compare(out, lse, c.want())
    # queries and outputs are device memory
    host = torch.empty(c.on["q"].shape, dtype=c.dt, pin_memory=True)
    for field in ("q", "out", "lse", "workspace"):
        old = getattr(a, field)
        setattr(a, field, host.data_ptr())
        if field != "workspace" or need.value:
            assert B.lib.hc_attend(c.pool.handle, ctypes.byref(a), None) == B.HC_ERR_INVALID
        setattr(a, field, old)
    c.close()


def test_store_and_page_calls_over_lists_in_pinned_memory():
    g = torch.Generator().manual_seed(3)
    dt = torch.bfloat16
    dev = [torch.zeros((1, 64, 64), dtype=dt, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    k = torch.randn((20, 1, 64), generator=g, dtype=torch.float64).to(dt).cuda()
    slots, pos = pinned(torch.randperm(64, generator=g)[:20]), pinned(torch.arange(20) * 100)
    rope = B.Rope(rot_dim=64)
    d = B.hc_store_desc(layer=0, dtype=B.HC_BF16, q_heads=0, kv_heads=1, head_dim=64, value_dim=64, n=20)
    d.slots, d.positions, d.k, d.v, d.rope = slots.data_ptr(), pos.data_ptr(), k.data_ptr(), k.data_ptr(), rope.handle.value
    d.k_stride[:] = d.v_stride[:] = (64, 64)
    torch.cuda.synchronize()
    assert B.lib.hc_store_tokens(pool.handle, ctypes.byref(d), None) == B.HC_OK
    torch.cuda.synchronize()
    y, s = F.rotate(k.cpu(), pos, F.frequencies(64, 10000.0), 1.0, 0, False)
    F.close(dev[0][0][slots.cuda()].view(20, 1, 64), y, s * 1.01 + F.half_step(dt) * y.abs(), "keys")
    assert torch.equal(F.bits(dev[1][0][slots.cuda()].view(20, 1, 64)), F.bits(k))
    table, lens = pinned(torch.tensor([[3, 1], [2, -1]])), pinned(torch.tensor([20, 16]))
    parents, free = pinned(torch.tensor([0, 1])), pinned(torch.tensor([0]))
    out, one = torch.zeros((2, 2), dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    before = [t.clone() for t in dev]
    assert B.lib.hc_fork_pages(pool.handle, table.data_ptr(), 2, 2, 2, lens.data_ptr(), parents.data_ptr(), 2,
                               free.data_ptr(), 1, out.data_ptr(), 2, one.data_ptr(), None) == B.HC_OK
    torch.cuda.synchronize()
    assert out.tolist() == [[3, 0], [2, -1]] and one.item() == 1
    for t, b in zip(dev, before):
        b[:, 0:4] = b[:, 16:20]
        assert torch.equal(F.bits(t), F.bits(b))
    work = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    pages = torch.zeros(4, dtype=torch.int64, device="cuda")
    assert B.lib.hc_free_pages(pool.handle, table.data_ptr(), 2, 2, 2, lens.data_ptr(), pages.data_ptr(), one.data_ptr(),
                               work.data_ptr(), 4096, None) == B.HC_OK
    torch.cuda.synchronize()
    assert one.item() == 1 and pages[0].item() == 0
    # what is written is device memory
    assert B.lib.hc_compact_pages(pool.handle, table.data_ptr(), 2, 2, 2, lens.data_ptr(), table.data_ptr(), 2,
                                  one.data_ptr(), work.data_ptr(), 4096, None) == B.HC_ERR_INVALID
    src, dst = pinned(torch.tensor([1])), pinned(torch.tensor([0]))
    assert B.lib.hc_copy_pages(pool.handle, src.data_ptr(), dst.data_ptr(), 1, None) == B.HC_OK
    torch.cuda.synchronize()
    pool.sync()
    assert torch.equal(F.bits(dev[0][:, :16]), F.bits(dev[0][:, 16:32]))
    pool.close()
