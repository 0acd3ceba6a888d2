"""Calls of the forward pass that are refused before anything is launched."""
import ctypes

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu


@pytest.fixture
def pool():
    dev = [torch.zeros((1, 64, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p = F.pool_of(dev, 16)
    yield p
    torch.cuda.synchronize()
    assert all(t.eq(0).all() for t in dev)
    p.sync()
    p.close()


def refused(rc, words):
    assert rc == B.HC_ERR_INVALID
    assert words in B.lib.hc_last_error().decode()


def test_strides_whose_products_pass_64_bits(pool):
    """Token strides of 2^40 elements over more than 2^22 rows: the extent is not the few bytes that
    it is modulo 2^64."""
    n = (1 << 22) + 1
    far = 1 << 40
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")  # padding: nothing would be read
    k = torch.zeros(256, dtype=torch.bfloat16, device="cuda")
    d = B.hc_store_desc(layer=0, dtype=B.HC_BF16, q_heads=0, kv_heads=2, head_dim=64, value_dim=64, n=n)
    d.slots, d.k, d.v = slots.data_ptr(), k.data_ptr(), k.data_ptr()
    d.k_stride[:], d.v_stride[:] = (far, 64), (0, 64)
    refused(B.lib.hc_store_tokens(pool.handle, ctypes.byref(d), None), "strides reach past")
    # a table of as many rows, each of length 0
    table = torch.zeros(4, dtype=torch.int64, device="cuda")
    lens = torch.zeros(n, dtype=torch.int64, device="cuda")
    pages, count = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    work = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    refused(B.lib.hc_free_pages(pool.handle, table.data_ptr(), n, 4, far, lens.data_ptr(), pages.data_ptr(),
                                count.data_ptr(), work.data_ptr(), 4096, None), "strides reach past")
    refused(B.lib.hc_compact_pages(pool.handle, table.data_ptr(), n, 4, far, lens.data_ptr(), table.data_ptr(), far,
                                   count.data_ptr(), work.data_ptr(), 4096, None), "strides reach past")
    refused(B.lib.hc_fork_pages(pool.handle, table.data_ptr(), n, 4, far, lens.data_ptr(), None, 0, None, 0, None, 4,
                                count.data_ptr(), None), "strides reach past")
    a = B.hc_attend_desc(layer=0, dtype=B.HC_BF16, q_heads=2, kv_heads=2, head_dim=64, value_dim=64, causal=1,
                         entry_tokens=16, scale=1.0, num_seqs=n, q_rows=1, max_q=1, max_kv=4, table_width=1,
                         table_stride=far)
    start = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    out = torch.zeros(128, dtype=torch.bfloat16, device="cuda")
    a.q, a.out, a.q_start, a.kv_len, a.table = (t.data_ptr() for t in (k, out, start, lens, table))
    a.q_stride[:] = a.out_stride[:] = (128, 64)
    refused(B.lib.hc_attend(pool.handle, ctypes.byref(a), None), "strides reach past")


def raises(call):
    with pytest.raises(B.HcError) as e:
        call()
    assert e.value.code == B.HC_ERR_INVALID and "overlap" in str(e.value), e.value


def test_attention_whose_outputs_overlap_what_it_reads(pool):
    """out over part of q, the lists, the layer's rows; lse and workspace over what is read or each other."""
    dt = torch.bfloat16
    raw = torch.zeros(1 << 16, dtype=dt, device="cuda")
    q = raw[:4 * 256].view(4, 4, 64)
    table = torch.zeros((1, 2), dtype=torch.int64, device="cuda")
    kv, start = torch.tensor([20]).cuda(), torch.tensor([0, 4]).cuda()

    def call(**kw):
        return pool.attend(0, kw.pop("q", q), kw.pop("table", table), kw.pop("kv_len", kv), kv_heads=2,
                           q_start=kw.pop("q_start", start), **kw)

    raises(lambda: call(out=raw[8:8 + 1024].view(4, 4, 64)))
    raises(lambda: call(out=raw[768:768 + 1024].view(4, 4, 64)))
    ints = raw.view(torch.int64)
    ints[:8] = 0
    raises(lambda: call(table=ints[16:18].view(1, 2), q=raw[4096:5120].view(4, 4, 64), out=q))
    raises(lambda: call(kv_len=ints[20:21], q=raw[4096:5120].view(4, 4, 64), out=q))
    raises(lambda: call(q_start=ints[255:257], q=raw[4096:5120].view(4, 4, 64), out=q))
    # the layer's own rows, as out and through the C call as lse and workspace
    view = pool.desc.sub[0].device_layers[0]
    d = B.hc_attend_desc(layer=0, dtype=B.HC_BF16, q_heads=4, kv_heads=2, head_dim=64, value_dim=64, causal=1,
                         entry_tokens=16, scale=1.0, num_seqs=1, q_rows=1, max_q=1, max_kv=20, table_width=2,
                         table_stride=2)
    out = torch.zeros((1, 4, 64), dtype=dt, device="cuda")
    work = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    d.q, d.out, d.kv_len, d.table, d.workspace = (t.data_ptr() for t in (q, out, kv, table, work))
    d.workspace_bytes = 1 << 20
    d.q_stride[:] = d.out_stride[:] = (256, 64)
    for field, at in [("out", view), ("lse", view), ("lse", q.data_ptr()), ("lse", out.data_ptr()),
                      ("lse", kv.data_ptr())]:
        old = getattr(d, field)
        setattr(d, field, at)
        refused(B.lib.hc_attend(pool.handle, ctypes.byref(d), None), "must not overlap")
        setattr(d, field, old)
    d.q_rows = d.num_seqs = 2  # two sequences of up to 512 slots may be split
    d.entry_tokens, d.table_width, d.table_stride, d.max_kv = 1, 512, 512, 512
    kv2, table2 = torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros((2, 512), dtype=torch.int64, device="cuda")
    out2, need = torch.zeros((2, 4, 64), dtype=dt, device="cuda"), ctypes.c_int64()
    d.kv_len, d.table, d.out = (t.data_ptr() for t in (kv2, table2, out2))
    assert B.lib.hc_attend_workspace_bytes(pool.handle, ctypes.byref(d), ctypes.byref(need)) == B.HC_OK
    assert 0 < need.value <= 1 << 20
    for field in ("q", "table", "out", "kv_len"):
        old = getattr(d, field)
        setattr(d, field, work.data_ptr() + 64)
        refused(B.lib.hc_attend(pool.handle, ctypes.byref(d), None), "must not overlap")
        setattr(d, field, old)


def test_store_whose_outputs_overlap_what_it_reads(pool):
    dt = torch.bfloat16
    raw = torch.zeros(1 << 14, dtype=dt, device="cuda")
    slots, n = torch.full((4,), -1, dtype=torch.int64, device="cuda"), 4
    q, k = raw[:1024].view(4, 4, 64), torch.zeros((4, 2, 64), dtype=dt, device="cuda")
    free = raw[8192:9216].view(4, 4, 64)
    raises(lambda: pool.store_tokens(0, slots, k, k, q=q, q_out=raw[8:1032].view(4, 4, 64)))
    raises(lambda: pool.store_tokens(0, slots, raw[1000:1512].view(4, 2, 64), k, q=free, q_out=q))
    raises(lambda: pool.store_tokens(0, slots, k, raw[1000:1512].view(4, 2, 64), q=free, q_out=q))
    rows = pool.desc.sub[0].device_layers[0]
    d = B.hc_store_desc(layer=0, dtype=B.HC_BF16, q_heads=0, kv_heads=2, head_dim=64, value_dim=64, n=n)
    d.slots, d.k, d.v = slots.data_ptr(), rows, k.data_ptr()
    d.k_stride[:] = d.v_stride[:] = (128, 64)
    refused(B.lib.hc_store_tokens(pool.handle, ctypes.byref(d), None), "must not overlap")
    d.k, d.v = k.data_ptr(), rows + 1024
    refused(B.lib.hc_store_tokens(pool.handle, ctypes.byref(d), None), "must not overlap")


def test_page_calls_whose_workspace_overlaps(pool):
    big = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    ints = big.view(torch.int64)
    table, lens = ints[:4].view(1, 4), torch.zeros(1, dtype=torch.int64, device="cuda")
    pages, count = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    args = (pool.handle, table.data_ptr(), 1, 4, 4, lens.data_ptr())
    refused(B.lib.hc_free_pages(*args, pages.data_ptr(), count.data_ptr(), big.data_ptr(), 4096, None), "overlaps")
    refused(B.lib.hc_compact_pages(*args, table.data_ptr(), 4, count.data_ptr(), big.data_ptr(), 4096, None), "overlaps")
    table = torch.zeros((1, 4), dtype=torch.int64, device="cuda")
    args = (pool.handle, table.data_ptr(), 1, 4, 4, lens.data_ptr())
    refused(B.lib.hc_free_pages(*args, ints[6:].data_ptr(), count.data_ptr(), big.data_ptr(), 4096, None), "overlaps")
    refused(B.lib.hc_free_pages(*args, pages.data_ptr(), ints[1:].data_ptr(), big.data_ptr(), 4096, None), "overlaps")
    refused(B.lib.hc_compact_pages(*args, table.data_ptr(), 4, ints[1:].data_ptr(), big.data_ptr(), 4096, None), "overlaps")


def test_views_between_each_other_are_no_overlap():
    """Queries, keys, values and outputs as views of one buffer: heads of a fused projection side by side and
    in turns, a table and its copy in one buffer."""
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(7)
    dev = [torch.zeros((1, 64, 128), dtype=dt, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    slots = torch.arange(40).cuda()
    table, lens = torch.arange(4).view(1, 4).cuda(), torch.tensor([40]).cuda()
    start = torch.tensor([0, 40]).cuda()
    for inner in (False, True):
        x = torch.randn((40, 2, 4, 64) if inner else (40, 4, 2, 64), generator=g, dtype=torch.float64).to(dt).cuda()
        q, k, v, out = (x[:, :, i] if inner else x[:, i] for i in range(4))
        plain = x.clone()
        pk, pv, pq = ((plain[:, :, i] if inner else plain[:, i]).contiguous() for i in (1, 2, 0))
        got = pool.store_tokens(0, slots, k, v, q=q, q_out=out)
        assert torch.equal(F.bits(got), F.bits(pq)) and got is out
        o, _ = pool.attend(0, q, table, lens, kv_heads=2, q_start=start, out=out)
        torch.cuda.synchronize()
        w, _, tol, _ = F.attend(pq.cpu(), pk.flatten(1).cpu(), pv.flatten(1).cpu(), torch.arange(40)[None], [40], [0, 40],
                                kv_heads=2, entry=1)
        F.close(out, w, tol, f"inner {inner}")
        for i, a in ((0, q), (1, k), (2, v)):
            assert torch.equal(F.bits(a), F.bits(plain[:, :, i] if inner else plain[:, i]))
    both = torch.full((3, 8), -9, dtype=torch.int64, device="cuda")
    both[:, :4] = torch.tensor([[3, 1, -1, -1], [2, -1, -1, -1], [-1, -1, -1, -1]])
    lens = torch.tensor([32, 5, 0]).cuda()
    assert pool.compact_pages(both[:, :4], lens, both[:, 4:]).item() == 3
    torch.cuda.synchronize()
    pool.sync()
    assert both[:, 4:].tolist() == [[0, 1, -1, -1], [2, -1, -1, -1], [-1, -1, -1, -1]]
    assert both[:, :4].tolist() == [[3, 1, -1, -1], [2, -1, -1, -1], [-1, -1, -1, -1]]
    pool.close()
