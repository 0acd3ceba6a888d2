"""Rows of a 4-bit cache on CPU tensors, from the definition, in 64 bits.  Test infrastructure."""
from __future__ import annotations

import torch

BLOCK = 32
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def row_bytes(heads, dim):
    n = heads * dim
    return (n // 2 + n // BLOCK + 15) // 16 * 16


def quantise(x):
    """(codes, scale bytes) of rows x (n, elements) of float64."""
    block = x.double().reshape(x.shape[0], -1, BLOCK)
    top = block.abs().amax(-1)
    bad = ~torch.isfinite(block).all(-1)
    top = torch.where(bad, 0.0, top)
    scale = torch.zeros(top.shape, dtype=torch.int64)
    for byte in range(254, -1, -1):  # the least power of two with the largest element within 7 of it
        scale = torch.where(top <= 7 * 2.0 ** (byte - 127), byte, scale)
    size = torch.where(bad[..., None], 0.0, block.abs()) / 2.0 ** (scale - 127).double()[..., None]
    # the nearest of the grid; of two equally near the one with the even code
    far = (size[..., None] - GRID).abs()
    near = far.amin(-1, keepdim=True)
    both = far == near
    codes = torch.arange(8)
    even = torch.where(both & (codes % 2 == 0), codes, -1).amax(-1)
    code = torch.where(even >= 0, even, both.int().argmax(-1))
    code = code + 8 * (torch.signbit(block) & ~bad[..., None]).long()
    scale = torch.where(bad, 255, scale)
    return code.reshape(x.shape[0], -1), scale


def pack(x, heads, dim, fill=0):
    """4-bit rows (n, bytes) of x (n, heads * dim); `fill`: the bytes behind the scales."""
    code, scale = quantise(x)
    n = heads * dim
    rows = torch.full((x.shape[0], row_bytes(heads, dim)), fill, dtype=torch.uint8)
    rows[:, :n // 2] = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    rows[:, n // 2:n // 2 + n // BLOCK] = scale.to(torch.uint8)
    return rows


def unpack(rows, heads, dim):
    """The values of 4-bit rows (..., bytes), in float64."""
    n = heads * dim
    byte = rows[..., :n // 2].long()
    code = torch.stack([byte % 16, byte // 16], -1).flatten(-2)
    value = torch.where(code >= 8, -GRID[code % 8], GRID[code % 8])
    scale = rows[..., n // 2:n // 2 + n // BLOCK].long()
    power = torch.where(scale == 255, torch.nan, 2.0 ** (scale - 127).double())
    return (value.unflatten(-1, (-1, BLOCK)) * power[..., None]).flatten(-2)
