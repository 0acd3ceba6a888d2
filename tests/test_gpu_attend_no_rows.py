"""Attention whose sequences have no rows, in a tensor of many: nothing is written, and nothing needs a workspace."""
import ctypes

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["elements", "mxfp4"])
@pytest.mark.parametrize("hq,hk,d", [(8, 8, 64), (8, 8, 128), (16, 1, 576)])
def test_a_bound_of_no_rows(hq, hk, d, cache):
    dt, n, page, dv = torch.bfloat16, 4500, 16, 512 if d == 576 else d
    row = M.row_bytes(hk, d) if cache == "mxfp4" else 2 * hk * d
    dev = [torch.zeros((1, 64 * page, row), dtype=torch.uint8, device="cuda") for _ in range(1 if d == 576 else 2)]
    pool = F.pool_of(dev, page)
    table = (torch.arange(n * 60) % 64).reshape(n, 60).cuda()
    q = torch.ones((n, hq, d), dtype=dt, device="cuda")
    start = torch.zeros(n + 1, dtype=torch.int64, device="cuda")
    kv = torch.full((n,), 900, device="cuda")
    desc = B.hc_attend_desc(layer=0, dtype=B.HC_BF16, q_heads=hq, kv_heads=hk, head_dim=d, value_dim=dv,
                            value_in_key=int(d != dv), causal=1, entry_tokens=page, scale=1.0, num_seqs=n, q_rows=n, max_q=0,
                            max_kv=900, table_width=60, table_stride=60)
    need = ctypes.c_int64(-1)
    size = B.lib.hc_attend_mxfp4_workspace_bytes if cache == "mxfp4" else B.lib.hc_attend_workspace_bytes
    assert size(pool.handle, ctypes.byref(desc), ctypes.byref(need)) == B.HC_OK and need.value == 0
    out = torch.full((n, hq, dv), 9.0, dtype=dt, device="cuda")

    def run():
        return pool.attend(0, q, table, kv, kv_heads=hk, q_start=start, max_q=0, max_kv=900, value_dim=dv, out=out, cache=cache)

    run()
    pool.sync()
    assert out.eq(9.0).all()
    start[7:] = 1  # a row after all: past the bound, and reported
    run()
    with pytest.raises(B.HcError, match="lengths out of bounds; first flagged list position 6"):
        pool.sync()
    assert out.eq(9.0).all()
    pool.close()
