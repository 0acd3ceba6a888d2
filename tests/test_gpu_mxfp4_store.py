"""Tokens stored into and fetched from a cache held in 4 bits, against the definition in 64 bits."""
import math

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M

pytestmark = pytest.mark.gpu


def pool_of(heads, dims, slots, page=16, layers=2, seed=0):
    """A pool of random bytes, so that what must stay can be told, and its buffers."""
    g = torch.Generator().manual_seed(seed)
    dev = [torch.randint(0, 256, (layers, slots, M.row_bytes(heads, d)), generator=g, dtype=torch.uint8).cuda() for d in dims]
    return F.pool_of(dev, page), dev


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_code_and_scale_fetched(dtype):
    """256 scales of 32 elements of every pair of codes."""
    dt = F.DTYPES[dtype]
    rows = torch.zeros((1, 256, 272), dtype=torch.uint8)
    rows[0, :, :256] = torch.arange(256, dtype=torch.uint8)  # 512 elements: every byte
    rows[0, :, 256:] = torch.arange(256, dtype=torch.uint8)[:, None]
    dev = rows.cuda()
    pool = F.pool_of([dev], 16)
    k = torch.empty((256, 4, 128), dtype=dt, device="cuda")
    pool.fetch_tokens(0, torch.arange(256, device="cuda"), k)
    want = M.unpack(rows[0], 4, 128).to(dt)  # rounded once; beyond the type infinite
    got = k.cpu().flatten(1)
    assert got.isnan().eq(want.isnan()).all()
    assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(want, 7.0))
    assert torch.equal(torch.signbit(got)[:255], torch.signbit(want)[:255])
    pool.sync()
    pool.close()


def edges(dt):
    """Rows of 64 whose elements lie on, just above and just below every border, at several sizes."""
    base = torch.tensor([0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 6.5], dtype=torch.float64)
    eps = torch.finfo(dt).eps
    x = torch.cat([base, base * (1 + 2 * eps), base * (1 - 2 * eps)])
    rows = []
    for e in (-8, -1, 0, 3, 12):
        for top in (4.0, 5.5, 6.0, 7.0, 7.0 * (1 + 2 * eps), 7.5):
            r = torch.zeros(64, dtype=torch.float64)
            r[:32], r[32:45] = x[:32], x[32:]
            r[1::2] *= -1
            r[31] = r[63] = top
            rows.append(r * 2.0 ** e)
    rows.append(torch.zeros(64, dtype=torch.float64))
    rows.append(torch.full((64,), -0.0, dtype=torch.float64))
    return torch.stack(rows).to(dt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_rounding(dtype):
    x = edges(F.DTYPES[dtype])
    n = len(x)
    pool, dev = pool_of(1, [64, 64], 64)
    before = [t.cpu() for t in dev]
    slots = torch.randperm(64, generator=torch.Generator().manual_seed(2))[:n]
    v = x.flip(0).contiguous()
    pool.store_tokens(1, slots.cuda(), x[:, None].cuda(), v[:, None].cuda(), cache="mxfp4")
    pool.sync()
    for t, was, y in zip(dev, before, (x, v)):
        was[1, slots, :34] = M.pack(y.double(), 1, 64)[:, :34]
        assert torch.equal(t.cpu(), was)
    pool.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_blocks_that_are_not_finite(dtype, value):
    dt = F.DTYPES[dtype]
    x = torch.ones((3, 2, 64), dtype=dt)
    x[0, 0, 3] = x[1, 1, 63] = value
    x[2, 0, 32:] = value
    pool, dev = pool_of(2, [64, 64], 16)
    slots = torch.tensor([5, 0, 9]).cuda()
    pool.store_tokens(0, slots, x.cuda(), x.cuda(), cache="mxfp4")
    k, v = torch.empty((2, 3, 2, 64), dtype=dt, device="cuda")
    pool.fetch_tokens(0, slots, k, v)
    want = torch.ones((3, 2, 64), dtype=dt)
    want[0, 0, :32] = want[1, 1, 32:] = want[2, 0, 32:] = math.nan
    for y in (k, v):
        assert torch.equal(torch.nan_to_num(y.cpu(), 9.0), torch.nan_to_num(want, 9.0))
    pool.sync()
    pool.close()


SHAPES = [dict(hq=8, hk=2, d=64, dv=64, rot=64), dict(hq=7, hk=1, d=128, dv=128, rot=32, offset=8),
          dict(hq=32, hk=8, d=128, dv=128, rot=128), dict(hq=3, hk=3, d=96, dv=32, rot=96, interleaved=True),
          dict(hq=0, hk=2, d=256, dv=64, rot=256), dict(hq=16, hk=1, d=576, dv=0, rot=64, offset=512, interleaved=True),
          dict(hq=4, hk=2, d=64, dv=64, rot=0), dict(hq=4, hk=1, d=64, dv=64, rot=16, offset=24),
          dict(hq=4, hk=2, d=128, dv=128, rot=128, sections=(16, 24, 24)),
          dict(hq=2, hk=2, d=64, dv=64, rot=64, pair_axes=[i % 2 for i in range(32)], interleaved=True)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(str(s[k]) for k in ("hq", "hk", "d", "dv", "rot")))
def test_rotated_and_stored(shape, n, dtype):
    dt = F.DTYPES[dtype]
    hq, hk, d, dv, rot = (shape[k] for k in ("hq", "hk", "d", "dv", "rot"))
    g = torch.Generator().manual_seed(n)
    S = 160
    pool, dev = pool_of(hk, [d] + ([dv] if dv else []), S)
    before = [t.cpu() for t in dev]

    def normal(*s):
        return torch.randn(s, generator=g, dtype=torch.float64).to(dt)

    q, k, v = normal(n, hq, d), normal(n, hk, d), normal(n, hk, dv)
    slots = torch.randperm(S, generator=g)[:n]
    offset, inter = shape.get("offset", 0), shape.get("interleaved", False)
    axes = {x: shape[x] for x in ("sections", "pair_axes") if x in shape}
    count = 1 + max(shape.get("pair_axes", [len(shape.get("sections", [0])) - 1]))
    pos = torch.randint(0, 100000, (count, n), generator=g)
    rope = B.Rope(rot_dim=rot, rot_offset=offset, interleaved=inter, base=10000.0, scaling="yarn", factor=4.0,
                  original_context=4096, **axes) if rot else None
    got_q = pool.store_tokens(1, slots.cuda(), k.cuda(), v.cuda() if dv else None, q=q.cuda() if hq else None, rope=rope,
                              positions=(pos if axes else pos[0]).cuda(), cache="mxfp4")
    pool.sync()
    yq, yk, sq = q.double(), k.double(), torch.zeros(q.shape, dtype=torch.float64)
    if rot:
        freq, magnitude = rope.frequencies()
        which = shape.get("pair_axes") or [a for a, c in enumerate(shape.get("sections", [rot // 2])) for _ in range(c)]
        yq, sq = rotate(q, pos, which, freq, magnitude, offset, inter)
        yk, _ = rotate(k, pos, which, freq, magnitude, offset, inter)
    if hq:
        F.close(got_q, yq, sq * 1.01 + F.half_step(dt) * yq.abs() + (2.0 ** -25 if dt == torch.float16 else 0.0), "queries")
    for t, was, y, e in zip(dev, before, (yk.flatten(1), v.double().flatten(1)), (d, dv)):
        here = hk * e // 2 + hk * e // 32
        want = M.pack(y, hk, e)
        got = t.cpu()
        # a border that the reference's own angle (53 bits, off by 2^-51 of position * f radians) cannot tell
        code, scale = M.quantise(y)
        unsure = near_border(y, hk * e, 1e-9 if e == d and rot else 0.0)
        mine = M.unpack(got[1][slots], hk, e)
        assert (torch.equal(got[1][slots][:, :here], want[:, :here]) or
                ((mine != M.unpack(want, hk, e)) <= unsure).all())
        got[1, slots, :here] = was[1, slots, :here]
        assert torch.equal(got, was)
    pool.close()


def near_border(y, elems, rel):
    """Elements whose code or block's scale would change by moving a value by `rel` of the block's largest."""
    block = y.reshape(len(y), -1, 32)
    top = block.abs().amax(-1, keepdim=True)
    lo, hi = M.quantise(y - rel * top.expand_as(block).reshape(y.shape)), M.quantise(y + rel * top.expand_as(block).reshape(y.shape))
    moved = (lo[0] != hi[0]) | (lo[1] != hi[1]).repeat_interleave(32, 1)
    return moved


def rotate(x, pos, which, freq, magnitude, offset, inter):
    """F.rotate with every pair at its axis' position: pairs of one axis at a time."""
    y, slack = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    for a in range(len(pos)):
        ya, sa = F.rotate(x, pos[a], freq, magnitude, offset, inter)
        for i, w in enumerate(which):
            if w == a:
                for e in ((offset + 2 * i, offset + 2 * i + 1) if inter else (offset + i, offset + len(which) + i)):
                    y[..., e], slack[..., e] = ya[..., e], sa[..., e]
    return y, slack


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 65])
@pytest.mark.parametrize("kw", [dict(sections=(16, 24, 24)), dict(sections=(40, 24), own_series=True),
                                dict(pair_axes=[i % 3 for i in range(64)])])
def test_axes_in_16_bits(kw, n, dtype):
    """A rope of several axes in the store of elements."""
    dt = F.DTYPES[dtype]
    g = torch.Generator().manual_seed(3)
    dev = [torch.zeros((1, 80, 256), dtype=dt, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    rope = B.Rope(rot_dim=128, base=10000.0, **kw)
    freq, magnitude = rope.frequencies()
    which = kw.get("pair_axes") or [a for a, c in enumerate(kw["sections"]) for _ in range(c)]
    q, k, v = (torch.randn((n, h, 128), generator=g, dtype=torch.float64).to(dt) for h in (6, 2, 2))
    pos = torch.randint(-5, 3000, (rope.axes, n), generator=g)
    slots = torch.randperm(80, generator=g)[:n]
    got = pool.store_tokens(0, slots.cuda(), k.cuda(), v.cuda(), q=q.cuda(), rope=rope, positions=pos.cuda())
    pool.sync()
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    for x, y in ((q, got), (k, dev[0][0][slots.cuda()].view(n, 2, 128))):
        want, slack = rotate(x, pos, which, freq, magnitude, 0, False)
        F.close(y, want, slack * 1.01 + F.half_step(dt) * want.abs() + tiny, "rotated")
    assert torch.equal(F.bits(dev[1][0][slots.cuda()].cpu().view(n, 2, 128)), F.bits(v))
    # axes that stand at one place rotate like one axis
    if not kw.get("own_series"):
        one = B.Rope(rot_dim=128, base=10000.0)
        a = pool.store_tokens(0, slots.cuda(), k.cuda(), v.cuda(), q=q.cuda(), rope=one, positions=pos[0].cuda().contiguous())
        b = pool.store_tokens(0, slots.cuda(), k.cuda(), v.cuda(), q=q.cuda(), rope=rope,
                              positions=pos[0].expand(rope.axes, n).contiguous().cuda())
        assert torch.equal(F.bits(a.cpu()), F.bits(b.cpu()))
    pool.close()


def test_padding_and_bad_slots():
    dt = torch.bfloat16
    pool, dev = pool_of(2, [64, 64], 32)
    before = [t.cpu() for t in dev]
    x = torch.randn((5, 2, 64), generator=torch.Generator().manual_seed(1)).to(dt).cuda()
    slots = torch.tensor([3, -1, 40, 7, -1]).cuda()
    q_out = torch.full((5, 2, 64), 5.0, dtype=dt, device="cuda")
    pool.store_tokens(0, slots, x, x, q=x, q_out=q_out, cache="mxfp4")
    with pytest.raises(B.HcError) as e:
        pool.sync()
    assert e.value.code == B.HC_ERR_DEVICE and "2" in str(e.value)
    for t, was in zip(dev, before):
        was[0, [3, 7], :68] = M.pack(x.cpu().double().flatten(1)[[0, 3]], 2, 64)[:, :68]
        assert torch.equal(t.cpu(), was)
    assert q_out[[1, 2, 4]].eq(5.0).all() and torch.equal(q_out[[0, 3]], x[[0, 3]])
    k = torch.full((5, 2, 64), 5.0, dtype=dt, device="cuda")
    v = k.clone()
    pool.fetch_tokens(0, slots, k, v)
    with pytest.raises(B.HcError) as e:
        pool.sync()
    assert e.value.code == B.HC_ERR_DEVICE and "2" in str(e.value)
    for y in (k, v):
        assert y[[1, 2, 4]].eq(5.0).all()
        assert torch.equal(y[[0, 3]].double().cpu().flatten(1), M.unpack(before[0][0, [3, 7]], 2, 64))
    pool.sync()
    pool.close()


def test_strides_and_broadcasts():
    """Tokens of a fused projection, one token for all, outputs between each other's rows."""
    dt = torch.float16
    g = torch.Generator().manual_seed(4)
    pool, dev = pool_of(2, [64, 64], 32)
    fused = torch.randn((6, 3, 2, 64), generator=g).to(dt).cuda()
    slots = torch.tensor([1, 30, 2, 9, 8, 31]).cuda()
    one = fused[:1, 2].expand(6, 2, 64)
    with pytest.raises(B.HcError):  # views of unlike token strides are told apart as a whole only
        pool.store_tokens(1, slots, fused[:, 0], one, q=fused[:, 1], q_out=fused[:, 1], cache="mxfp4")
    one = one[:1].clone().expand(6, 2, 64)
    q = pool.store_tokens(1, slots, fused[:, 0], one, q=fused[:, 1], q_out=fused[:, 1], cache="mxfp4")
    both = torch.zeros((6, 2, 2, 64), dtype=dt, device="cuda")
    pool.fetch_tokens(1, slots, both[:, :, 0], both[:, :, 1])
    want = [M.unpack(M.pack(y.cpu().double().flatten(1), 2, 64), 2, 64) for y in (fused[:, 0], one)]
    for i in range(2):
        assert torch.equal(both[:, :, i].double().cpu().flatten(1), want[i])
    assert q.data_ptr() == fused[:, 1].data_ptr()
    pool.sync()
    pool.close()


def test_refusals():
    dt = torch.bfloat16
    pool, dev = pool_of(2, [64, 64], 32)
    x = torch.zeros((4, 2, 64), dtype=dt, device="cuda")
    slots = torch.arange(4, device="cuda")
    for call, code in [
        (lambda: pool.store_tokens(0, slots, x, x), B.HC_ERR_INVALID),                       # rows of 16 bits
        (lambda: pool.store_tokens(0, slots, x[:, :1], x[:, :1], cache="mxfp4"), B.HC_ERR_INVALID),
        (lambda: pool.store_tokens(0, slots, x[..., :48], x[..., :48], cache="mxfp4"), B.HC_ERR_UNSUPPORTED),
        (lambda: pool.store_tokens(2, slots, x, x, cache="mxfp4"), B.HC_ERR_INVALID),
        (lambda: pool.fetch_tokens(2, slots, x, x.clone()), B.HC_ERR_INVALID),
        (lambda: pool.fetch_tokens(0, slots, x, x), B.HC_ERR_INVALID),                       # k over v
        (lambda: pool.fetch_tokens(0, slots, x[:1].expand(4, 2, 64), x.clone()), B.HC_ERR_INVALID),
        (lambda: pool.fetch_tokens(0, slots, x[..., :48], x[..., 48:]), B.HC_ERR_UNSUPPORTED),
        (lambda: pool.fetch_tokens(0, x.view(torch.int64).flatten()[:4], x, x.clone()), B.HC_ERR_INVALID),
        (lambda: pool.fetch_tokens(0, slots, dev[0].view(torch.bfloat16).flatten()[:512].view(4, 2, 64)), B.HC_ERR_INVALID),
    ]:
        with pytest.raises(B.HcError) as e:
            call()
        assert e.value.code == code, e.value
    with pytest.raises(ValueError):
        pool.store_tokens(0, slots, x, x, cache="int4")
    with pytest.raises(ValueError):
        pool.store_tokens(0, slots, x, x, rope=B.Rope(rot_dim=64, sections=(16, 16)), positions=slots, cache="mxfp4")
    with pytest.raises(ValueError):
        pool.store_tokens(0, slots, x, x, rope=B.Rope(rot_dim=64, sections=(16, 16)),
                          positions=torch.zeros((4, 2), dtype=torch.int64, device="cuda"), cache="mxfp4")
    pool.store_tokens(0, slots[:0], x[:0], x[:0], cache="mxfp4")
    pool.fetch_tokens(0, slots[:0], x[:0])
    pool.sync()
    pool.close()


def test_captured_and_on_another_stream():
    dt = torch.bfloat16
    g = torch.Generator().manual_seed(5)
    pool, dev = pool_of(2, [64, 64], 32)
    rope = B.Rope(rot_dim=64, sections=(8, 24))
    x = torch.randn((6, 2, 64), generator=g).to(dt).cuda()
    slots, pos = torch.zeros(6, dtype=torch.int64, device="cuda"), torch.zeros((2, 6), dtype=torch.int64, device="cuda")
    k, v = torch.empty((2, 6, 2, 64), dtype=dt, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pool.store_tokens(1, slots, x, x, rope=rope, positions=pos, cache="mxfp4")
        pool.fetch_tokens(1, slots, k, v)
    for i in range(4):
        slots.copy_(torch.randperm(32, generator=g)[:6])
        pos.copy_(torch.randint(0, 1000, (2, 6), generator=g))
        x.copy_(torch.randn((6, 2, 64), generator=g).to(dt))
        graph.replay()
        torch.cuda.synchronize()
        got = k.clone(), v.clone()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        pool.store_tokens(0, slots, x, x, rope=rope, positions=pos, cache="mxfp4", stream=other)
        pool.fetch_tokens(0, slots, k, v, stream=other)
        other.synchronize()
        assert torch.equal(got[0], k) and torch.equal(got[1], v) and k.ne(0).any()
        assert torch.equal(dev[0][0][slots][:, :68], dev[0][1][slots][:, :68])
    pool.sync()
    del graph
    pool.close()
