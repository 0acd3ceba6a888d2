"""Plain 64-bit implementations of the forward-pass operators on CPU tensors, pools to run the
library's on, and the error bounds that the comparison uses.  Test infrastructure."""
from __future__ import annotations

import math

import torch

from host_device_page_amd import binding as B

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def pool_of(buffers, page, blocks=(), stream=None, flags=0):
    """A device-only pool over (layers, slots or pages, elements) tensors; those whose place is
    in `blocks` hold page blocks."""
    layers = buffers[0].shape[0]
    slots = next(t.shape[1] for i, t in enumerate(buffers) if i not in blocks)
    subs = [(B.HC_PAGE_BLOCKS if i in blocks else B.HC_TOKEN_ROWS, t.shape[2] * t.element_size())
            for i, t in enumerate(buffers)]
    return B.Pool(layers=layers, page_size=page, subs=subs, device_slots=slots, host_pages=0,
                  device_layers=[[t[i] for i in range(layers)] for t in buffers], host=None, stream=stream, flags=flags)


def frequencies(rot, base, scaling="none", factor=1.0, original=0, low=1.0, high=4.0, fast=32.0, slow=1.0):
    """Radians per position of each pair, from the definitions, pair by pair."""
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling == "llama3":
        out = []
        for x in f:
            turns = original * x / (2 * math.pi)
            if turns < low:
                x = x / factor
            elif turns <= high:
                s = (turns - low) / (high - low)
                x = (1 - s) * x / factor + s * x
            out.append(x)
        return out
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(rot // 2)]
        return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]
    return f


def rotate(x, positions, freq, magnitude, rot_offset, interleaved):
    """(value, bound without the final rounding) of rotated heads x (n, heads, dim)."""
    f = torch.tensor(freq, dtype=torch.float64)
    # angles as fractions of a turn by exact integers: position * f / 2 pi, f's own 53 bits
    angle = positions.double()[:, None] * f[None]
    c, s = torch.cos(angle)[:, None] * magnitude, torch.sin(angle)[:, None] * magnitude
    y, slack = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64)
    h = len(freq)
    a = slice(rot_offset, rot_offset + 2 * h, 2) if interleaved else slice(rot_offset, rot_offset + h)
    b = slice(rot_offset + 1, rot_offset + 2 * h, 2) if interleaved else slice(rot_offset + h, rot_offset + 2 * h)
    x1, x2 = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    # fp32: the angle's fraction is rounded to 24 bits (pi * 2^-25), sine and cosine to a few
    # units, three roundings follow: below 16 units of 2^-24 on |x1| + |x2|
    slack[..., a] = slack[..., b] = 16 * U32 * magnitude * (x1.abs() + x2.abs())
    # far positions: this reference's own 53-bit angle
    slack[..., a] += (x1.abs() + x2.abs()) * magnitude * (positions.double().abs()[:, None] * f * 2.0 ** -51)[:, None]
    slack[..., b] = slack[..., a]
    return y, slack


def slots_of(table_row, kv, entry):
    j = torch.arange(kv)
    return table_row[j // entry] * entry + j % entry


def seen(position, keys, causal, window, sinks):
    if not causal:
        return torch.ones(len(keys), dtype=torch.bool)
    ok = keys <= position
    if window:
        ok = ok & ((position - keys < window) | (keys < sinks))
    return ok


def attend(q, k_rows, v_rows, table, kv_len, q_start, *, kv_heads, entry, causal=True, window=0, sinks=0, scale=None,
           value_dim=None, hidden=()):
    """(out, lse, bound of out, bound of lse): 64 bits, row by row; rows of no sequence are NaN
    in `out`.  k_rows, v_rows: (slots, elements); v_rows None: the head of the key rows.
    hidden: (sequence, key) pairs that a bad table entry hides."""
    rows, heads, dim = q.shape
    dv = value_dim or dim
    group = heads // kv_heads
    scale = dim ** -0.5 if scale is None else scale
    u = half_step(q.dtype)
    out = torch.full((rows, heads, dv), math.nan, dtype=torch.float64)
    lse = torch.full((rows, heads), math.nan, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for s in range(len(kv_len)):
        kv, a, b = int(kv_len[s]), int(q_start[s]), int(q_start[s + 1])
        where = slots_of(table[s].clamp(min=0), kv, entry) if kv else torch.zeros(0, dtype=torch.int64)
        keys = torch.arange(kv)
        there = torch.ones(kv, dtype=torch.bool)
        for seq, key in hidden:
            if seq == s:
                there[key] = False
        k = k_rows[where].double().view(kv, kv_heads, dim)
        v = k[..., :dv] if v_rows is None else v_rows[where].double().view(kv, kv_heads, dv)
        for r in range(a, b):
            ok = seen(kv - (b - a) + r - a, keys, causal, window, sinks) & there
            for h in range(heads):
                kk, vv, x = k[ok, h // group], v[ok, h // group], q[r, h].double()
                score = (kk * x).sum(-1) * scale
                top = score.max() if len(score) else torch.tensor(-math.inf)
                if len(score) == 0 or top == -math.inf:
                    out[r, h], lse[r, h] = 0.0, -math.inf
                    continue
                e = torch.exp(score - top)
                p = e / e.sum()
                out[r, h] = (p[:, None] * vv).sum(0)
                lse[r, h] = top + e.sum().log()
                # a score is `dim` products and sums in fp32 (any order), the scale, and the
                # exponential's argument and result: relative error of each weight.  The sum over
                # keys may drop low bits of n terms.
                mag = (kk.abs() * x.abs()).sum(-1).max().item() * abs(scale)
                n = len(score)
                d = (dim + 8) * U32 * mag + 8 * U32 * (score.abs().max().item() + 4)
                spread = (p[:, None] * vv.abs()).sum(0)
                # weights as operands: one rounding each; fp16 ones below its normal range are off
                # by half of its smallest step, relative to a largest weight of 1
                tiny = n * 2.0 ** -25 * vv.abs().amax(0) if q.dtype == torch.float16 else 0.0
                tol[r, h] = u * out[r, h].abs() + (1 + u) * ((u + 2 * d + 2 * (n + 16) * U32) * spread + tiny)
                if q.dtype == torch.float16:
                    tol[r, h] += 2.0 ** -25
                tol_lse[r, h] = d + (n + 16) * U32 + 4 * U32 * lse[r, h].abs()
    return out, lse, tol, tol_lse


def close(got, want, tol, what):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, what
    same = (got == want) | (got.isnan() & want.isnan())
    ok = same | ((got - want).abs() <= tol)
    if not bool(ok.all()):
        bad = (~ok).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {len(bad)} of {ok.numel()} values off, first {i}: got {got[i].item()!r}, want "
                             f"{want[i].item()!r}, bound {tol[i].item() if torch.is_tensor(tol) else tol!r}")


def bits(t):
    return t.contiguous().view(torch.int16)
