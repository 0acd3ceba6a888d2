"""Attention with scales at and next to zero over scores as large as fp32 holds."""
import pytest
import torch

from tests import forward_support as F
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu

# query rows of the two sequences: decoding tiles and many rows; latent rows up to 16, up to 32 and more
HEADS = [(64, 2, 4, (1, 1)), (64, 2, 4, (30, 33)), (128, 2, 4, (1, 1)), (128, 2, 4, (40, 3)), (576, 1, 4, (1, 1)),
         (576, 1, 20, (1, 1)), (576, 1, 4, (40, 9))]


@pytest.mark.parametrize("scale", [0.0, 1e-38, -1e-38, 3e-38])
@pytest.mark.parametrize("d,hk,hq,q", HEADS)
def test_scales_next_to_zero(d, hk, hq, q, scale):
    """Queries and keys whose products are near 2^126: a scale of 0 weighs all keys alike, and scales down
    to fp32's least normal numbers weigh them by what is left."""
    c = Case(hq=hq, hk=hk, d=d, kv=(150, 70), q=q, page=16)
    size = {64: 60, 128: 59, 576: 58}[d]  # d * 2^(2 size) stays below 2^127
    g = torch.Generator().manual_seed(d)
    c.q = torch.full_like(c.q, 2.0 ** size)
    keys = c.host[0][c.layer]
    keys[:, :] = 2.0 ** size * (torch.randint(0, 5, (len(keys), 1), generator=g) - 2) / 2
    c.upload().check(scale=scale)
    c.close()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,hk,hq,q", HEADS)
def test_small_weights_of_many_keys(d, hk, hq, q, dtype):
    """One key of a large score and no value, the others of weights next to 2^-16, below fp16's normal range: what
    they add up to is the output."""
    c = Case(dtype=dtype, hq=hq, hk=hk, d=d, kv=(1500, 700), q=q, page=16)
    c.q.zero_()
    c.q[..., d - 1] = 1.0
    keys, values = c.host[0][c.layer], c.host[-1][c.layer]
    keys.zero_()
    if d == 576:
        keys.view(len(keys), hk, d)[..., :512] = 1.0
    else:
        values[:] = 1.0
    first = [F.slots_of(c.table[s], 1, c.entry) for s in range(2)]
    for where in first:
        keys[where] = 0.0
        keys.view(len(keys), hk, d)[where, :, d - 1] = 11.0625
        if d != 576:
            values[where] = 0.0
    c.upload()
    out, lse = c.run(scale=1.0)
    torch.cuda.synchronize()
    want = c.want(scale=1.0)
    assert want[0].gt(0.009).all()
    c.compare(out, lse, want)
    c.close()
