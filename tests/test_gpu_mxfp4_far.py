"""Rows of a 4-bit cache whose offsets pass 32 bits: stored, fetched, attended to, and copied."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hk,d,q_len", [(8, 128, 1), (8, 128, 40), (1, 576, 1), (1, 576, 20), (1, 576, 130)])
def test_rows_behind_4_gib(hk, d, q_len):
    dt, P, hq = torch.bfloat16, 16, 8 if hk == 8 else 4
    latent = d == 576
    dv = 512 if latent else d
    row = B.mxfp4_row_bytes(hk, d)
    pages = (1 << 32) // (row * P) + 60
    dev = [torch.zeros((1, pages * P, row), dtype=torch.uint8, device="cuda") for _ in range(1 if latent else 2)]
    pool = F.pool_of(dev, P)
    g = torch.Generator().manual_seed(1)
    kv = 200 if q_len < 100 else 150
    used = -(-kv // P)
    far = torch.randperm(50, generator=g)[:used] + pages - 50
    table = far[None].cuda()
    slots = F.slots_of(far, kv, P)
    assert int(slots.min()) * row > 1 << 32
    k, v = (torch.randn((kv, hk, d), generator=g).to(dt) for _ in range(2))
    pool.store_tokens(0, slots.cuda(), k.cuda(), None if latent else v.cuda(), cache="mxfp4")
    back = [torch.empty((kv, hk, d), dtype=dt, device="cuda") for _ in dev]
    pool.fetch_tokens(0, slots.cuda(), *back)
    rows = [M.unpack(M.pack(x.double().flatten(1), hk, d), hk, d) for x in (k, v)[:len(dev)]]
    for x, y in zip(back, rows):
        assert torch.equal(x.cpu().double().flatten(1), y)
    q = torch.randn((q_len, hq, d), generator=g).to(dt)
    start = torch.tensor([0, q_len])
    out, _ = pool.attend(0, q.cuda(), table, torch.tensor([kv]).cuda(), kv_heads=hk, q_start=start.cuda(), max_kv=kv,
                         value_dim=dv, cache="mxfp4")
    near = torch.arange(used)[None]  # the same rows, packed
    packed = [torch.cat([y, torch.zeros(used * P - kv, hk * d)]).to(dt) for y in rows]
    w, _, tol, _ = F.attend(q, packed[0], None if latent else packed[1], near, [kv], start.tolist(), kv_heads=hk, entry=P,
                            value_dim=dv)
    F.close(out, w, tol, "out")
    pool.copy_pages(far[:1].cuda(), torch.tensor([3]).cuda())
    pool.sync()
    for t in dev:
        assert torch.equal(t[0, 3 * P:4 * P], t[0, int(far[0]) * P:(int(far[0]) + 1) * P]) and t[0, :3 * P].eq(0).all()
    pool.close()
