"""Ropes of several axes and the 4-bit cache's entry points without a GPU: frequencies, sizes, and the
refusals that come before any device is touched."""
import ctypes
import math

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M

AXES = dict(rot_dim=64, rot_offset=0, interleaved=0, scaling=B.HC_ROPE_NONE, base=1e4, factor=1.0, low_freq_factor=1.0,
            high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0, magnitude=0.0, original_context=4096)


def create(pair_axes, axes, own_series=0, **kw):
    out = ctypes.c_void_p(1)
    pairs = None if pair_axes is None else (ctypes.c_int32 * len(pair_axes))(*pair_axes)
    rc = B.lib.hc_rope_create_axes(ctypes.byref(B.hc_rope_desc(**dict(AXES, **kw))), pairs, axes, own_series,
                                   ctypes.byref(out))
    if rc == B.HC_OK:
        assert B.lib.hc_rope_destroy(out) == B.HC_OK
    else:
        assert out.value is None
    return rc


def test_axes_refusals():
    good = [i % 3 for i in range(32)]
    assert create(good, 3) == B.HC_OK
    assert create(good, 3, 1) == B.HC_OK
    assert create(None, 1) == B.HC_OK
    for pairs, axes in [(None, 2), (good, 2), (good, 4), (good, 0), (good, 9), ([-1] + good[1:], 3), (good, -1)]:
        assert create(pairs, axes) == B.HC_ERR_INVALID, axes
    assert create(good, 3, rot_dim=24) == B.HC_ERR_UNSUPPORTED
    assert B.lib.hc_rope_create_axes(None, None, 1, 0, None) == B.HC_ERR_INVALID


def test_axes_share_one_series():
    want, _ = B.Rope(rot_dim=128, base=1e6, scaling="yarn", factor=4.0, original_context=4096).frequencies()
    for kw in (dict(sections=(16, 24, 24)), dict(pair_axes=[i % 3 for i in range(64)])):
        r = B.Rope(rot_dim=128, base=1e6, scaling="yarn", factor=4.0, original_context=4096, **kw)
        assert r.axes == 3 and r.frequencies()[0] == want


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="llama3", factor=8.0, original=8192),
                                dict(scaling="yarn", factor=4.0, original=4096)])
def test_axes_with_series_of_their_own(kw):
    """Every axis like a rotation of twice its pairs."""
    r = B.Rope(rot_dim=96, base=1e4, sections=(8, 16, 24), own_series=True, scaling=kw.get("scaling", "none"),
               factor=kw.get("factor", 1.0), original_context=kw.get("original", 0))
    got = r.frequencies()[0]
    at = 0
    for n in (8, 16, 24):
        for g, w in zip(got[at:at + n], F.frequencies(2 * n, 1e4, **kw)):
            assert math.isclose(g, w, rel_tol=1e-13)
        at += n
    # the same axes in turns: the j-th pair of an axis, wherever it is
    order = [0] * 8 + [1] * 16 + [2] * 24
    mixed = order[::-1]
    turned = B.Rope(rot_dim=96, base=1e4, pair_axes=mixed, own_series=True, scaling=kw.get("scaling", "none"),
                    factor=kw.get("factor", 1.0), original_context=kw.get("original", 0)).frequencies()[0]
    assert [x for a in range(3) for x, m in zip(turned, mixed) if m == a] == got


def test_axes_arguments():
    with pytest.raises(ValueError):
        B.Rope(rot_dim=64, sections=(16, 15))
    with pytest.raises(ValueError):
        B.Rope(rot_dim=64, sections=(16, 16), pair_axes=[0] * 32)
    with pytest.raises(ValueError):
        B.Rope(rot_dim=64, own_series=True)
    with pytest.raises(B.HcError):
        B.Rope(rot_dim=64, sections=(32, 0))
    assert B.Rope(rot_dim=64).axes == 1


@pytest.mark.parametrize("heads,dim", [(1, 64), (8, 128), (1, 576), (4, 96), (2, 32), (16, 256)])
def test_row_bytes(heads, dim):
    assert B.mxfp4_row_bytes(heads, dim) == M.row_bytes(heads, dim)


def test_row_bytes_refusals():
    n = ctypes.c_int64()
    for heads, dim, code in [(0, 64, B.HC_ERR_INVALID), (1, 0, B.HC_ERR_INVALID), (1, 40, B.HC_ERR_UNSUPPORTED)]:
        assert B.lib.hc_mxfp4_row_bytes(heads, dim, ctypes.byref(n)) == code
    assert B.lib.hc_mxfp4_row_bytes(1, 64, None) == B.HC_ERR_INVALID


def test_null_arguments():
    n = ctypes.c_int64()
    assert B.lib.hc_store_tokens_mxfp4(None, None, None) == B.HC_ERR_INVALID
    assert B.lib.hc_fetch_tokens_mxfp4(None, None, None) == B.HC_ERR_INVALID
    assert B.lib.hc_attend_mxfp4(None, None, None) == B.HC_ERR_INVALID
    assert B.lib.hc_attend_mxfp4_workspace_bytes(None, None, ctypes.byref(n)) == B.HC_ERR_INVALID
    assert B.lib.hc_extend_pages(None, None, None) == B.HC_ERR_INVALID


def test_rows_of_the_definition():
    """The reference itself: what is stored is read as it is, no element off by more than half a step, the scale the
    least that allows it."""
    x = torch.randn((50, 64), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    x[0] = 0
    x[1, :32] = 7.0
    x[2, 5] = math.inf
    rows = M.pack(x, 1, 64)
    y = M.unpack(rows, 1, 64)
    assert torch.equal(M.pack(torch.where(y.isnan(), math.nan, y), 1, 64)[3:], rows[3:])
    assert y[0].eq(0).all() and y[1, :32].eq(6).all() and y[2, :32].isnan().all() and y[2, 32:].isfinite().all()
    step = 2.0 ** (rows[:, 32:34].long() - 127).double().repeat_interleave(32, 1)
    a = x.abs() / step
    half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0)) * step
    ok = y.isfinite()
    assert ((x - y).abs() <= half)[ok].all()
    top = (x.abs() / step).unflatten(1, (2, 32)).amax(-1)
    assert ((top > 3.5) & (top <= 7))[3:].all()
