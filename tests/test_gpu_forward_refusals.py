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
