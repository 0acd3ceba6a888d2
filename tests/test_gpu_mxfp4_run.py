"""The operators of a 4-bit cache together, as a serving step uses them: pages for a batch's new tokens, rotated with several
axes and stored, attended to, written back, loaded into other pages, decoded, forked and packed."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M

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

    row = B.mxfp4_row_bytes(hk, d)
    subs = [(B.HC_TOKEN_ROWS, row)] * (1 if latent else 2)
    dev = [torch.zeros((L, S, row), dtype=torch.uint8, device="cuda") for _ in subs]
    host = B.HostBuffer(L * S * sum(e for _, e in subs))
    copy = torch.cuda.Stream()
    pool = B.Pool(layers=L, page_size=P, subs=subs, device_slots=S, host_pages=pages,
                  device_layers=[[t[l] for l in range(L)] for t in dev], host=host, stream=copy)
    rope = B.Rope(rot_dim=64, rot_offset=512 if latent else 0, interleaved=latent, base=10000.0, sections=(8, 12, 12))

    def rows(i, l, wide):
        return M.unpack(dev[i][l].cpu(), hk, wide).to(dt)

    def attended(l, q, table, lens, q_start, out, what):
        w, _, tol, _ = F.attend(q.cpu(), rows(0, l, d), None if latent else rows(1, l, dv), table.cpu(), lens, q_start,
                                kv_heads=hk, entry=P, value_dim=dv)
        F.close(out, w, tol, what)

    # two prompts into an empty pool
    table = torch.full((2, 6), -1, dtype=torch.int64, device="cuda")
    none = torch.zeros(2, dtype=torch.int64, device="cuda")
    free, n_free = pool.free_pages(table, none)
    assert n_free.item() == pages
    free = free[torch.randperm(pages, generator=g).cuda()]
    added = torch.tensor([37, 64], device="cuda")
    lens, q_start, slots, pos, used = pool.extend_pages(table, none, added, free, tokens=101)
    assert lens.tolist() == [37, 64] and used.item() == 7 and table[0, :3].tolist() == free[:3].tolist()
    first = used.clone()
    axes = torch.stack([pos, pos // 7, pos % 7])
    outs = []
    for l in range(L):
        q, k, v = normal(101, hq, d), normal(101, hk, d), normal(101, hk, dv)
        q_rot = pool.store_tokens(l, slots, k, None if latent else v, q=q, rope=rope, positions=axes, cache="mxfp4")
        back = torch.empty_like(k), None if latent else torch.empty_like(v)
        pool.fetch_tokens(l, slots, *back)
        assert torch.equal(back[0].cpu().flatten(1), rows(0, l, d)[slots.cpu()])
        if not latent:
            assert torch.equal(dev[1][l][slots].cpu()[:, :136], M.pack(v.cpu().double().flatten(1), hk, dv)[:, :136])
        out, _ = pool.attend(l, q_rot, table, lens, kv_heads=hk, q_start=q_start, value_dim=dv, cache="mxfp4")
        attended(l, q_rot, table, lens.tolist(), q_start.tolist(), out, f"layer {l}")
        outs.append((q_rot, out))
    # to the host and back into other pages
    stored = torch.cuda.Event()
    stored.record()
    copy.wait_event(stored)
    whole = torch.cat([table[0, :3], table[1, :4]])
    d_idx = (whole[:, None] * P + torch.arange(P, device="cuda")).flatten()
    h_idx = torch.arange(7 * P) + 5 * P
    pool.write_back_all_layers(d_idx, h_idx)
    new = free[7:14]
    n_idx = (new[:, None] * P + torch.arange(P, device="cuda")).flatten()
    h_dev = h_idx.cuda()
    events = [B.HipEvent() for _ in range(L)]
    torch.cuda.current_stream().synchronize()
    for l in range(L):
        pool.load_back_layer(l, h_dev, n_idx, events[l])
    table[0, :3], table[1, :4] = new[:3], new[3:]
    first += 7
    for l in range(L):  # each layer as soon as it has arrived
        events[l].wait_on(torch.cuda.current_stream())
        q_rot, out = outs[l]
        again, _ = pool.attend(l, q_rot, table, lens, kv_heads=hk, q_start=q_start, value_dim=dv, cache="mxfp4")
        assert torch.equal(F.bits(again), F.bits(out)), l
    # branch five samples, and decode a token of each: the second prompt ended at a page's end
    parents = torch.tensor([0, 0, 1, 0, 0], device="cuda")
    child = torch.full((5, 6), -1, dtype=torch.int64, device="cuda")
    taken = pool.fork_pages(table, lens, parents, free[14:].contiguous(), child)
    assert taken.item() == 4
    first += taken
    ones = torch.ones(5, dtype=torch.int64, device="cuda")
    kv, start, at, where, used = pool.extend_pages(child, lens[parents].contiguous(), ones, free, tokens=5, first_free=first)
    assert used.item() == 1 and kv.tolist() == [38, 38, 65, 38, 38] and where.tolist() == [37, 37, 64, 37, 37]
    q, k, v = normal(5, hq, d), normal(5, hk, d), normal(5, hk, dv)
    q_rot = pool.store_tokens(1, at, k, None if latent else v, q=q, rope=rope, positions=where.expand(3, 5).contiguous(),
                              cache="mxfp4")
    out, _ = pool.attend(1, q_rot, child, kv, kv_heads=hk, value_dim=dv, cache="mxfp4")
    attended(1, q_rot, child, kv.tolist(), start.tolist(), out, "decode on forks")
    # the parents are gone: pack what the children hold, and decode once more
    packed = torch.empty_like(child)
    count = pool.compact_pages(child, kv, packed)
    assert count.item() == 2 + 4 + 4 + 1
    again, _ = pool.attend(1, q_rot, packed, kv, kv_heads=hk, value_dim=dv, cache="mxfp4")
    assert torch.equal(F.bits(again), F.bits(out))
    pool.sync()
    pool.close()
    host.free()


def test_a_step_in_one_graph():
    """Pages, store and attention of a decoding step captured once, and replayed as the sequences grow."""
    dt = torch.bfloat16
    P, pages, hq, hk, d = 4, 64, 8, 2, 64
    row = B.mxfp4_row_bytes(hk, d)
    dev = [torch.zeros((1, pages * P, row), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, P)
    rope = B.Rope(rot_dim=64)
    g = torch.Generator().manual_seed(2)
    free = torch.randperm(pages, generator=g).cuda()
    table = torch.full((3, 12), -1, dtype=torch.int64, device="cuda")
    lens, first = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    ones = torch.ones(3, dtype=torch.int64, device="cuda")
    q, k, v = (torch.zeros((4, h, d), dtype=dt, device="cuda") for h in (hq, hk, hk))  # a row of padding
    out = torch.full((4, hq, d), 9.0, dtype=dt, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        kv, start, slots, pos, used = pool.extend_pages(table, lens, ones, free, tokens=4, first_free=first)
        q_rot = pool.store_tokens(0, slots, k, v, q=q, rope=rope, positions=pos, cache="mxfp4")
        pool.attend(0, q_rot, table, kv, kv_heads=hk, q_start=start, max_q=1, max_kv=48, out=out, cache="mxfp4")
        lens.copy_(kv)
        first += used
    for step in range(1, 10):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g).to(dt))
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [step] * 3 and first.item() == 3 * -(-step // P) and slots[3] == -1
        w, _, tol, _ = F.attend(q_rot[:3].cpu(), M.unpack(dev[0][0].cpu(), hk, d).to(dt), M.unpack(dev[1][0].cpu(), hk, d).to(dt),
                                table.cpu(), [step] * 3, [0, 1, 2, 3], kv_heads=hk, entry=P)
        F.close(out[:3], w, tol, f"step {step}")
        assert out[3].eq(9.0).all()
    pool.sync()
    del graph
    pool.close()
