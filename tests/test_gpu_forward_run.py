"""The operators together, as a serving step uses them: store, attend, write back, load back into
other slots, attend there, fork, decode on the forks, compact, decode again."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("latent", [False, True])
def test_a_serving_run(latent):
    dt = torch.bfloat16
    L, P, pages, hq = 3, 16, 48, 8
    hk, d, dv = (1, 576, 512) if latent else (2, 128, 128)
    S = P * pages
    g = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64).to(dt).cuda()

    dev = [torch.zeros((L, S, hk * e), dtype=dt, device="cuda") for e in ([d] if latent else [d, dv])]
    subs = [(B.HC_TOKEN_ROWS, hk * e * 2) for e in ([d] if latent else [d, dv])]
    host = B.HostBuffer(L * S * sum(e for _, e in subs))
    copy = torch.cuda.Stream()
    pool = B.Pool(layers=L, page_size=P, subs=subs, device_slots=S, host_pages=pages,
                  device_layers=[[t[l] for l in range(L)] for t in dev], host=host, stream=copy)
    rope = B.Rope(rot_dim=64, rot_offset=512 if latent else 0, interleaved=latent, base=10000.0)
    freq, magnitude = rope.frequencies()
    lens = [37, 64]
    place = torch.randperm(pages, generator=g)
    table = torch.full((2, 6), -1, dtype=torch.int64)
    table[0, :3], table[1, :4] = place[:3], place[3:7]
    slots = torch.cat([F.slots_of(table[s], n, P) for s, n in enumerate(lens)])
    pos = torch.cat([torch.arange(n) for n in lens])
    q_start = torch.tensor([0, 37, 101])
    n = 101
    rows = [[], []]   # what each layer's rows should hold, from 64 bits
    outs = []
    for l in range(L):
        q, k, v = normal(n, hq, d), normal(n, hk, d), normal(n, hk, dv)
        q_rot = pool.store_tokens(l, slots.cuda(), k, None if latent else v, q=q, rope=rope, positions=pos.cuda())
        out, _ = pool.attend(l, q_rot, table.cuda(), torch.tensor(lens).cuda(), kv_heads=hk, q_start=q_start.cuda(),
                             value_dim=dv)
        y, slack = F.rotate(k.cpu(), pos, freq, magnitude, 512 if latent else 0, latent)
        F.close(dev[0][l][slots.cuda()].view(n, hk, d), y, slack * 1.01 + F.half_step(dt) * y.abs(), "keys")
        w, _, tol, _ = F.attend(q_rot.cpu(), dev[0][l].cpu(), None if latent else dev[1][l].cpu(), table, lens, q_start,
                                kv_heads=hk, entry=P, value_dim=dv)
        F.close(out, w, tol, f"layer {l}")
        outs.append((q_rot, out))
    # to the host and back into other pages
    stored = torch.cuda.Event()
    stored.record()
    copy.wait_event(stored)
    whole = [int(x) for x in table[0, :3]] + [int(x) for x in table[1, :4]]
    d_idx = torch.cat([torch.arange(P) + p * P for p in whole])
    h_idx = torch.arange(7 * P) + 5 * P
    pool.write_back_all_layers(d_idx.cuda(), h_idx)
    new = place[7:14]
    n_idx = torch.cat([torch.arange(P) + int(p) * P for p in new])
    events = [B.HipEvent() for _ in range(L)]
    h_dev, n_dev = h_idx.cuda(), n_idx.cuda()
    torch.cuda.current_stream().synchronize()
    moved = torch.full((2, 6), -1, dtype=torch.int64)
    moved[0, :3], moved[1, :4] = new[:3], new[3:]
    on, ln = moved.cuda(), torch.tensor(lens).cuda()
    for l in range(L):
        pool.load_back_layer(l, h_dev, n_dev, events[l])
    for l in range(L):  # each layer as soon as it has arrived
        events[l].wait_on(torch.cuda.current_stream())
        q_rot, out = outs[l]
        again, _ = pool.attend(l, q_rot, on, ln, kv_heads=hk, q_start=q_start.cuda(), value_dim=dv)
        assert torch.equal(F.bits(again), F.bits(out)), l
    # fork: four samples of the first, one of the second; they decode one token each
    free, n_free = pool.free_pages(on, ln)
    parents = torch.tensor([0, 0, 1, 0, 0]).cuda()
    child = torch.empty((5, 6), dtype=torch.int64, device="cuda")
    used = pool.fork_pages(on, ln, parents, free[:n_free.item()].contiguous(), child)
    assert used.item() == 4
    child_len = ln[parents]
    # the second's child ends at a page border: its next token needs a page of its own
    child[2, 4] = free[4]
    at = child.gather(1, (child_len // P)[:, None])[:, 0] * P + child_len % P
    q, k, v = normal(5, hq, d), normal(5, hk, d), normal(5, hk, dv)
    q_rot = pool.store_tokens(1, at, k, None if latent else v, q=q, rope=rope, positions=child_len)
    out, _ = pool.attend(1, q_rot, child, child_len + 1, kv_heads=hk, value_dim=dv)
    w, _, tol, _ = F.attend(q_rot.cpu(), dev[0][1].cpu(), None if latent else dev[1][1].cpu(), child.cpu(),
                            (child_len + 1).tolist(), list(range(6)), kv_heads=hk, entry=P, value_dim=dv)
    F.close(out, w, tol, "decode on forks")
    # the parents are gone: pack what the children hold, and decode once more
    packed = torch.empty_like(child)
    count = pool.compact_pages(child, child_len + 1, packed)
    assert count.item() == 2 + 4 + 4 + 1
    again, _ = pool.attend(1, q_rot, packed, child_len + 1, kv_heads=hk, value_dim=dv)
    assert torch.equal(F.bits(again), F.bits(out))
    pool.sync()
    pool.close()
    host.free()
