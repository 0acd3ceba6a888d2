"""Tokens of a 4-bit cache at the ends of their element type, against the definition in 64 bits."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M

pytestmark = pytest.mark.gpu


def held(y, dt, heads, dim):
    """4-bit rows of y (n, heads * dim) in 64 bits, read as float64: M.quantise's, but an element below the power of two behind
    `dt`'s largest value, whose code stands for more than dt holds, takes the largest code that dt holds."""
    code, scale = M.quantise(y)
    most = torch.finfo(dt).max
    behind = 2.0 ** (16 if dt == torch.float16 else 128)
    power = 2.0 ** (scale - 127).double().repeat_interleave(M.BLOCK, 1)
    for _ in range(7):  # from code to code
        over = (y.abs() < behind) & (M.GRID[code % 8] * power > most)
        code = torch.where(over, code - 1, code)
    rows = torch.zeros((len(y), M.row_bytes(heads, dim)), dtype=torch.uint8)
    n = heads * dim
    rows[:, :n // 2] = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    rows[:, n // 2:n // 2 + n // M.BLOCK] = scale.to(torch.uint8)
    return rows


def largest(dt):
    """Rows of 64 around the type's largest values: every one of them the largest of a block, and each beside larger ones."""
    ints = torch.int16
    top = torch.tensor([torch.finfo(dt).max], dtype=dt).view(ints).item()
    values = torch.arange(top - 700, top + 1, dtype=ints).view(dt)  # fp16 from 43600, bf16 from 1.1 * 2^122
    g = torch.Generator().manual_seed(1)
    x = torch.randn((len(values) + 64, 64), generator=g, dtype=torch.float64) * (torch.finfo(dt).max / 16)
    x = x.to(dt)
    x[:len(values), 5] = values
    x[:len(values), 40] = -values
    x[len(values):] = values[torch.randint(0, len(values), (64, 64), generator=g)]
    x[len(values)::2, ::2] *= -1
    return x


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_largest_elements_are_stored_finite(dtype):
    dt = F.DTYPES[dtype]
    x = largest(dt)
    assert x.isfinite().all()
    n = len(x)
    dev = [torch.zeros((1, -(-n // 16) * 16, 48), dtype=torch.uint8, device="cuda") for _ in range(2)]
    pool = F.pool_of(dev, 16)
    slots = torch.randperm(n, generator=torch.Generator().manual_seed(2))
    v = x.flip(0).contiguous()
    pool.store_tokens(0, slots.cuda(), x[:, None].cuda(), v[:, None].cuda(), cache="mxfp4")
    k_out, v_out = torch.empty((2, n, 1, 64), dtype=dt, device="cuda")
    pool.fetch_tokens(0, slots.cuda(), k_out, v_out)
    pool.sync()
    for t, y, back in zip(dev, (x, v), (k_out, v_out)):
        rows = t.cpu()[0, slots]
        assert back.isfinite().all()
        assert torch.equal(rows[:, :34], held(y.double(), dt, 1, 64)[:, :34])
        assert torch.equal(back.cpu()[:, 0].double(), M.unpack(rows, 1, 64))
    pool.close()


def test_rotated_keys_past_the_type():
    """Of fp16 tokens, turned and stretched to 2^16 and more: those are what their codes stand for, and infinite as fp16; elements
    of their blocks that fp16 holds stay finite."""
    dt = torch.float16
    n = 400
    g = torch.Generator().manual_seed(3)
    x = torch.randn((n, 64), generator=g, dtype=torch.float64) * 2.0 ** torch.randint(8, 16, (n, 1), generator=g)
    x = x.clamp(-65504, 65504).to(dt)
    rope = B.Rope(rot_dim=64, magnitude=24.0)  # position 0: every element times 24, exactly
    dev = [torch.zeros((1, 400, 48), dtype=torch.uint8, device="cuda")]
    pool = F.pool_of(dev, 16)
    slots = torch.arange(n).cuda()
    pool.store_tokens(0, slots, x[:, None].cuda(), rope=rope, positions=torch.zeros_like(slots), cache="mxfp4")
    back = torch.empty((n, 1, 64), dtype=dt, device="cuda")
    pool.fetch_tokens(0, slots, back)
    pool.sync()
    y = x.double() * 24
    top = M.quantise(y)[1]
    assert all((top == byte).any() for byte in (140, 141, 142, 143, 144, 145))  # every case was met
    rows = held(y, dt, 1, 64)
    assert torch.equal(dev[0].cpu()[0][:, :34], rows[:, :34])
    assert back.cpu()[:, 0].isfinite()[y.abs() < 2 ** 16].all()
    assert torch.equal(back.cpu()[:, 0], M.unpack(rows, 1, 64).to(dt))
    pool.close()


# bf16 values of this size would pass fp32 in a sum over keys, whose weights are relative to about the largest
@pytest.mark.parametrize("dtype,large", [("bf16", "keys"), ("fp16", "keys"), ("fp16", "values")])
@pytest.mark.parametrize("d,q", [(64, (1, 3)), (128, (70, 1)), (576, (1, 2)), (576, (40, 1))])
def test_attention_over_the_largest_elements(d, q, dtype, large):
    """Keys, or values, up to the type's largest; of a latent cache the elements that are only key, or also value."""
    dt = F.DTYPES[dtype]
    g = torch.Generator().manual_seed(d)
    latent = d == 576
    hk, hq, dv, kv, page = (1, 16, 512, (90, 60), 16) if latent else (2, 4, d, (90, 60), 16)
    n = sum(kv)

    def normal(*shape):
        return torch.randn(shape, generator=g, dtype=torch.float64).to(dt)

    def most(*shape):
        x = (torch.rand(shape, generator=g, dtype=torch.float64) * 0.2 + 0.8) * torch.finfo(dt).max
        x = (x * torch.randint(0, 2, shape, generator=g).mul(2).sub(1)).to(dt)
        assert x.isfinite().all()
        return x

    k, v, x = normal(n, hk, d), normal(n, hk, dv), normal(sum(q), hq, d)
    scale = None
    if large == "keys":
        scale = 1.0 / (torch.finfo(dt).max / 64)  # scores, sums of products in fp32 with queries of up to 1/8, of about 1
        x = (x.double() / 64).to(dt)
        if latent:
            k[..., dv:] = most(n, hk, d - dv)
        else:
            k = most(n, hk, d)
    elif latent:
        k[..., :dv] = most(n, hk, dv)
        x[..., :dv] = 0.0  # (else one key would have all the weight)
    else:
        v = most(n, hk, dv)
    table = torch.tensor([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, -1, -1]])
    slots = torch.cat([F.slots_of(table[s], m, page) for s, m in enumerate(kv)])
    dev = [torch.zeros((1, 160, M.row_bytes(hk, e)), dtype=torch.uint8, device="cuda") for e in ([d] if latent else [d, d])]
    pool = F.pool_of(dev, page)
    pool.store_tokens(0, slots.cuda(), k.cuda(), None if latent else v.cuda(), cache="mxfp4")
    start = torch.tensor([0, q[0], sum(q)])
    out, lse = pool.attend(0, x.cuda(), table.cuda(), torch.tensor(kv).cuda(), kv_heads=hk, q_start=start.cuda(), max_q=max(q),
                           max_kv=max(kv), value_dim=dv, return_lse=True, scale=scale, cache="mxfp4")
    pool.sync()
    rows = [M.unpack(t[0].cpu(), hk, e).to(dt) for t, e in zip(dev, (d, dv))]
    w, wl, tol, tol_l = F.attend(x, rows[0], None if latent else rows[1], table, kv, start.tolist(), kv_heads=hk, entry=page,
                                 value_dim=dv, scale=scale)
    assert w.isfinite().all() and out.isfinite().all()
    F.close(out, w, tol, "out")
    F.close(lse, wl, tol_l, "lse")
    pool.close()
