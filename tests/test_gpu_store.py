"""Rotary positions and the store of new tokens, against 64 bits."""
import math

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu


def made(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(dtype)


CASES = [
    # tokens, q heads, kv heads, head, value, rope
    dict(n=1, hq=32, hk=8, d=128, dv=128, rope=dict(rot=128, base=500000.0, scaling="llama3", factor=8.0, original=8192)),
    dict(n=37, hq=6, hk=2, d=64, dv=64, rope=dict(rot=32, base=10000.0)),
    dict(n=5, hq=7, hk=1, d=96, dv=96, rope=dict(rot=96, base=10000.0, scaling="linear", factor=3.0), interleaved=True),
    dict(n=33, hq=16, hk=1, d=576, dv=0, rope=dict(rot=64, base=10000.0, scaling="yarn", factor=40.0, original=4096),
         offset=512, interleaved=True),
    dict(n=3, hq=2, hk=2, d=256, dv=40, rope=dict(rot=256, base=10000.0)),
    dict(n=4100, hq=4, hk=4, d=64, dv=64, rope=dict(rot=64, base=10000.0)),  # several tokens a workgroup
    dict(n=9, hq=0, hk=3, d=64, dv=64, rope=dict(rot=16, base=10000.0), offset=24),
    dict(n=9, hq=4, hk=2, d=8, dv=8, rope=None),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("ci", range(len(CASES)))
def test_store_against_64_bits(ci, dtype):
    c, dt = CASES[ci], F.DTYPES[dtype]
    n, hq, hk, d, dv = (c[k] for k in ("n", "hq", "hk", "d", "dv"))
    S, L = n + 23, 3
    host = [made((L, S, hk * e), dt, 10 + i) for i, e in enumerate([d] + ([dv] if dv else []))]
    k, v, q = made((n, hk, d), dt, 1), made((n, hk, dv), dt, 2) if dv else None, made((n, hq, d), dt, 3) if hq else None
    g = torch.Generator().manual_seed(4)
    slots = torch.randperm(S, generator=g)[:n]
    positions = torch.randint(0, 1 << 20, (n,), generator=g)
    positions[0] = (1 << 31) + 12345
    slots[n // 2] = -1 if n > 1 else slots[0]  # a padding token
    dev = [t.cuda() for t in host]
    pool = F.pool_of(dev, 1)
    rope = None
    if c["rope"]:
        r = c["rope"]
        rope = B.Rope(rot_dim=r["rot"], base=r["base"], scaling=r.get("scaling", "none"), factor=r.get("factor", 1.0),
                      original_context=r.get("original", 0), rot_offset=c.get("offset", 0),
                      interleaved=c.get("interleaved", False))
    q_out = torch.full((n, hq, d), 7.0, dtype=dt, device="cuda") if hq else None
    got = pool.store_tokens(1, slots.cuda(), k.cuda(), v.cuda() if dv else None, q=q.cuda() if hq else None,
                            q_out=q_out, rope=rope, positions=positions.cuda())
    torch.cuda.synchronize()
    pool.sync()
    keep = slots >= 0
    u = F.half_step(dt)

    def turned(x):
        if not c["rope"]:
            return x.double(), torch.zeros(x.shape, dtype=torch.float64)
        m = 0.1 * math.log(c["rope"]["factor"]) + 1 if c["rope"].get("scaling") == "yarn" else 1.0
        y, slack = F.rotate(x, positions, F.frequencies(**c["rope"]), m, c.get("offset", 0), c.get("interleaved", False))
        # one rounding of what is rotated, off by half a step (fp16: of its smallest step at least)
        off = slack * (1 + u) + u * y.abs() * (slack > 0) + (2.0 ** -25 if dt == torch.float16 else 0.0) * (slack > 0)
        return y, off

    want, tol = [t.double() for t in host], [torch.zeros(t.shape, dtype=torch.float64) for t in host]
    y, off = turned(k)
    want[0][1, slots[keep]], tol[0][1, slots[keep]] = y[keep].flatten(1), off[keep].flatten(1)
    if dv:
        want[1][1, slots[keep]] = v[keep].double().flatten(1)
    for i in range(len(host)):  # every other row and layer as it was
        F.close(dev[i], want[i], tol[i], f"sub {i}")
    if hq:
        assert got is q_out
        y, off = turned(q)
        y[~keep], off[~keep] = 7.0, 0.0
        F.close(got, y, off, "q")
    pool.close()


def test_fused_rows_in_place_and_payload_bits():
    """q, k, v as views of one projection, queries rotated in place; values (NaN payloads,
    infinities) move bit for bit; k's heads broadcast by a stride of 0."""
    n, hq, hk, d = 21, 4, 2, 64
    dt = torch.bfloat16
    rows = made((n, hq + 2 * hk, d), dt, 5).cuda()
    rows[:, hq + hk:] = torch.randint(-32768, 32768, (n, hk, d), dtype=torch.int16).view(dt).cuda()
    dev = [torch.zeros((1, 64, hk * d), dtype=dt, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    rope = B.Rope(rot_dim=64)
    slots, pos = torch.arange(n).cuda() + 3, torch.arange(n).cuda() * 1000
    q, k, v = rows[:, :hq], rows[:, hq:hq + 1].expand(n, hk, d), rows[:, hq + hk:]
    before = rows.clone()
    pool.store_tokens(0, slots, k, v, q=q, q_out=q, rope=rope, positions=pos)
    torch.cuda.synchronize()
    f = F.frequencies(64, 10000.0)
    y, s = F.rotate(before[:, :hq].cpu(), pos.cpu(), f, 1.0, 0, False)
    F.close(q, y, s * 1.01 + F.half_step(dt) * y.abs(), "q in place")
    y, s = F.rotate(before[:, hq:hq + 1].expand(n, hk, d).cpu(), pos.cpu(), f, 1.0, 0, False)
    F.close(dev[0][0, 3:3 + n].view(n, hk, d), y, s * 1.01 + F.half_step(dt) * y.abs(), "k")
    assert torch.equal(F.bits(dev[1][0, 3:3 + n].view(n, hk, d)), F.bits(before[:, hq + hk:]))
    assert torch.equal(F.bits(rows[:, hq:]), F.bits(before[:, hq:]))
    pool.close()


def test_far_positions_keep_their_angle():
    """Positions whose fp32 angle would be off by turns: exact rational angles from integers."""
    d, n = 64, 6
    pos = torch.tensor([0, 1, -5, 10 ** 7 + 1, (1 << 40) + 3, (1 << 52) + 1])
    x = torch.zeros((n, 1, d), dtype=torch.float16)
    x[..., :32] = 1.0
    dev = [torch.zeros((1, 16, d), dtype=torch.float16, device="cuda")]
    pool = F.pool_of(dev, 1)
    rope = B.Rope(rot_dim=64, base=10000.0)
    pool.store_tokens(0, torch.arange(n).cuda(), x.cuda(), rope=rope, positions=pos.cuda())
    got = dev[0][0, :n].cpu().double()
    from fractions import Fraction
    freq = rope.frequencies()[0]
    # pi to 60 digits
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    for i in range(n):
        for p in range(32):
            turns = Fraction(freq[p]) * int(pos[i]) / (2 * pi)
            a = float((turns - (turns.numerator // turns.denominator)) * 2 * pi)
            # the table's own rounding: 2^-65 of a turn per position
            off = abs(int(pos[i])) * 2.0 ** -64 * 2 * math.pi + 16 * F.U32 + 2.0 ** -11
            assert abs(got[i, p] - math.cos(a)) <= off and abs(got[i, 32 + p] - math.sin(a)) <= off, (i, p)
    pool.close()


def test_bad_slots_are_skipped_and_reported():
    dt = torch.bfloat16
    dev = [torch.zeros((2, 16, 64), dtype=dt, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    k = torch.ones((4, 1, 64), dtype=dt, device="cuda")
    q_out = torch.full((4, 1, 64), 5.0, dtype=dt, device="cuda")
    pool.store_tokens(0, torch.tensor([3, 16, -2, 1 << 40]).cuda(), k, k, q=k, q_out=q_out)
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="out of range; first flagged list position 1"):
        pool.sync()
    pool.sync()  # cleared
    assert dev[0][0, 3].eq(1).all() and dev[0].sum() == 64 and dev[1].sum() == 64
    assert q_out[0].eq(1).all() and q_out[1:].eq(5).all()
    pool.store_tokens(1, torch.empty(0, dtype=torch.int64).cuda(), k[:0], k[:0])  # no token
    pool.sync()
    pool.close()


def test_refusals():
    dt = torch.bfloat16
    dev = [torch.zeros((1, 16, 128), dtype=dt, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    slots, k = torch.arange(4).cuda(), torch.ones((4, 2, 64), dtype=dt, device="cuda")
    rope = B.Rope(rot_dim=64, rot_offset=8)

    def refuse(code, *a, **kw):
        with pytest.raises(B.HcError) as e:
            pool.store_tokens(*a, **kw)
        assert e.value.code == code, e.value

    refuse(B.HC_ERR_INVALID, 1, slots, k, k)                           # no such layer
    refuse(B.HC_ERR_INVALID, 0, slots, k[:, :1], k[:, :1])             # rows of another size
    refuse(B.HC_ERR_INVALID, 0, slots, k, k, rope=rope, positions=slots)  # rotates past the head
    wide = torch.ones((4, 2, 68), dtype=dt, device="cuda")
    refuse(B.HC_ERR_UNSUPPORTED, 0, slots, wide[..., :64], k)          # stride 68
    refuse(B.HC_ERR_UNSUPPORTED, 0, slots, wide.view(-1)[4:4 + 512].view(4, 2, 64), k)  # 8-byte aligned
    q = torch.ones((4, 1, 64), dtype=dt, device="cuda")
    refuse(B.HC_ERR_INVALID, 0, slots, k, k, q=q, q_out=q[:1].expand(4, 1, 64))  # outputs overlap
    with pytest.raises(TypeError):
        pool.store_tokens(0, slots, k.float(), k.float())
    with pytest.raises(TypeError):
        pool.store_tokens(0, slots.int(), k, k)
    with pytest.raises(ValueError):
        pool.store_tokens(0, slots[:3], k, k)
    assert dev[0].eq(0).all() and dev[1].eq(0).all()
    pool.close()
