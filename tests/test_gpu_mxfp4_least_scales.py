"""4-bit blocks of the least scales, whose borders are subnormal fp32 numbers, against the definition in 64 bits."""
import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M

pytestmark = pytest.mark.gpu

BORDERS = torch.tensor([0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0], dtype=torch.float64)


def stored(x, **kw):
    """Rows of 64 elements x (n, 64), stored and read back: their bytes, and the elements."""
    n = len(x)
    dev = [torch.zeros((1, n, 48), dtype=torch.uint8, device="cuda")]
    pool = F.pool_of(dev, 1)
    slots = torch.arange(n).cuda()
    pool.store_tokens(0, slots, x[:, None].cuda(), cache="mxfp4",
                      **{k: torch.zeros_like(slots) if v is None else v for k, v in kw.items()})
    back = torch.empty((n, 1, 64), dtype=x.dtype, device="cuda")
    pool.fetch_tokens(0, slots, back)
    pool.sync()
    pool.close()
    return dev[0].cpu()[0][:, :34], back.cpu()[:, 0]


def test_every_small_element():
    """All bf16 magnitudes from 0 to 2^-116, beside others of their size and alone with a larger one."""
    ints = torch.arange(0, 11 * 128, dtype=torch.int16)
    near = ints.view(torch.bfloat16).reshape(-1, 64)  # 2^-133 to 2^-116, 64 neighbours a row
    alone = torch.zeros((len(ints), 64), dtype=torch.bfloat16)
    alone[:, 7] = -ints.view(torch.bfloat16)
    alone[:, 40] = ints.view(torch.bfloat16)
    alone[:, 60] = (BORDERS * 2.0 ** -127)[torch.arange(len(ints)) % len(BORDERS)].to(torch.bfloat16)
    g = torch.Generator().manual_seed(1)
    mixed = ints[torch.randint(0, len(ints), (500, 64), generator=g)].view(torch.bfloat16)
    mixed = torch.where(torch.rand(mixed.shape, generator=g) < 0.5, mixed, -mixed)
    x = torch.cat([near, -near, alone, mixed])
    rows, back = stored(x)
    want = M.pack(x.double(), 1, 64)[:, :34]
    assert (want[:, 32:] == 0).any() and (want[:, 32:] == 9).any()
    assert torch.equal(rows, want)
    assert torch.equal(back.double(), M.unpack(want, 1, 64))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("e", [-127, -126, -125, -124, -20, 0, 100])
def test_rotated_keys_next_to_borders(e, interleaved):
    """Elements on a border times 1 - 2^-40 and 1 + 2^-40: less from it than fp32 can tell, on the side that 64 bits say."""
    x = BORDERS.repeat(5)[:64].repeat(15, 1)
    x = x * torch.arange(64).remainder(3).sub(0.5).sign()
    x[:, 1::2] = x[:, 1::2].flip(1)
    x[:, 31] = x[:, 63] = BORDERS  # the largest of a block on every border too, where smaller ones allow it
    for r in range(15):
        x[r] = torch.where(x[r].abs() <= BORDERS[r], x[r], BORDERS[r] / 4)
    x = torch.cat([x, BORDERS.repeat(5)[:64][None].expand(2, 64)])
    x[-1, 31] = x[-1, 63] = 4.0
    x = (x * 2.0 ** e).to(torch.bfloat16)
    for magnitude in (1 - 2.0 ** -40, 1 + 2.0 ** -40):
        rope = B.Rope(rot_dim=64, magnitude=magnitude, interleaved=interleaved)  # at position 0: nothing is turned
        rows, _ = stored(x, rope=rope, positions=None)
        assert torch.equal(rows, M.pack(x.double() * magnitude, 1, 64)[:, :34]), magnitude
