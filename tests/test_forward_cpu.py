"""The forward-pass entry points without a GPU: rotary frequencies, and the refusals that
come before any device is touched."""
import ctypes
import math

import pytest

from host_device_page_amd import binding as B
from tests import forward_support as F


@pytest.mark.parametrize("kw", [
    dict(rot=128, base=10000.0),
    dict(rot=16, base=500000.0),
    dict(rot=64, base=10000.0, scaling="linear", factor=4.0),
    dict(rot=128, base=500000.0, scaling="llama3", factor=8.0, original=8192),
    dict(rot=96, base=10000.0, scaling="llama3", factor=32.0, original=2048, low=2.0, high=9.0),
    dict(rot=64, base=10000.0, scaling="yarn", factor=40.0, original=4096),
    dict(rot=256, base=1000000.0, scaling="yarn", factor=4.0, original=32768, fast=16.0, slow=2.0),
    dict(rot=32, base=10000.0, scaling="yarn", factor=2.0, original=8),  # every pair turns slowly
])
def test_frequencies(kw):
    r = B.Rope(rot_dim=kw["rot"], base=kw["base"], scaling=kw.get("scaling", "none"), factor=kw.get("factor", 1.0),
               original_context=kw.get("original", 0), low_freq_factor=kw.get("low", 1.0),
               high_freq_factor=kw.get("high", 4.0), beta_fast=kw.get("fast", 32.0), beta_slow=kw.get("slow", 1.0))
    got, magnitude = r.frequencies()
    want = F.frequencies(**kw)
    assert len(got) == kw["rot"] // 2
    # exp and pow in doubles: a few units of 2^-53, times the exponent's own rounding
    for g, w in zip(got, want):
        assert math.isclose(g, w, rel_tol=1e-13)
    yarn = 0.1 * math.log(kw["factor"]) + 1 if kw.get("scaling") == "yarn" else 1.0
    assert math.isclose(magnitude, yarn, rel_tol=1e-15)


def test_given_magnitude():
    assert B.Rope(rot_dim=16, magnitude=0.25).frequencies()[1] == 0.25


GOOD = dict(rot_dim=64, rot_offset=0, interleaved=0, scaling=B.HC_ROPE_NONE, base=1e4, factor=1.0, low_freq_factor=1.0,
            high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0, magnitude=0.0, original_context=4096)


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), B.HC_ERR_INVALID),
    (dict(rot_dim=24), B.HC_ERR_UNSUPPORTED),
    (dict(rot_dim=272), B.HC_ERR_INVALID),
    (dict(rot_offset=-8), B.HC_ERR_INVALID),
    (dict(rot_offset=4), B.HC_ERR_UNSUPPORTED),
    (dict(scaling=9), B.HC_ERR_INVALID),
    (dict(base=1.0), B.HC_ERR_INVALID),
    (dict(base=math.inf), B.HC_ERR_INVALID),
    (dict(base=math.nan), B.HC_ERR_INVALID),
    (dict(scaling=B.HC_ROPE_LINEAR, factor=0.0), B.HC_ERR_INVALID),
    (dict(scaling=B.HC_ROPE_YARN, factor=math.nan), B.HC_ERR_INVALID),
    (dict(magnitude=-1.0), B.HC_ERR_INVALID),
    (dict(scaling=B.HC_ROPE_LLAMA3, high_freq_factor=1.0), B.HC_ERR_INVALID),
    (dict(scaling=B.HC_ROPE_LLAMA3, original_context=0), B.HC_ERR_INVALID),
    (dict(scaling=B.HC_ROPE_YARN, beta_slow=0.0), B.HC_ERR_INVALID),
    (dict(scaling=B.HC_ROPE_YARN, beta_fast=0.5), B.HC_ERR_INVALID),
])
def test_rope_refusals(kw, code):
    d = B.hc_rope_desc(**dict(GOOD, **kw))
    out = ctypes.c_void_p(1)
    assert B.lib.hc_rope_create(ctypes.byref(d), ctypes.byref(out)) == code
    assert out.value is None


def test_rope_accepts_the_good_one():
    out = ctypes.c_void_p()
    assert B.lib.hc_rope_create(ctypes.byref(B.hc_rope_desc(**GOOD)), ctypes.byref(out)) == B.HC_OK
    assert B.lib.hc_rope_destroy(out) == B.HC_OK


def test_null_arguments():
    n, f = ctypes.c_int64(), ctypes.c_double()
    assert B.lib.hc_rope_create(None, None) == B.HC_ERR_INVALID
    assert B.lib.hc_rope_destroy(None) == B.HC_OK
    assert B.lib.hc_rope_frequencies(None, ctypes.byref(f), ctypes.byref(f)) == B.HC_ERR_INVALID
    assert B.lib.hc_store_tokens(None, None, None) == B.HC_ERR_INVALID
    assert B.lib.hc_attend(None, None, None) == B.HC_ERR_INVALID
    assert B.lib.hc_attend_workspace_bytes(None, None, ctypes.byref(n)) == B.HC_ERR_INVALID
    assert B.lib.hc_copy_pages(None, None, None, 0, None) == B.HC_ERR_INVALID
    assert B.lib.hc_fork_pages(None, None, 0, 0, 0, None, None, 0, None, 0, None, 0, None, None) == B.HC_ERR_INVALID
    assert B.lib.hc_pages_workspace_bytes(None, ctypes.byref(n)) == B.HC_ERR_INVALID
    assert B.lib.hc_free_pages(None, None, 0, 0, 0, None, None, None, None, 0, None) == B.HC_ERR_INVALID
    assert B.lib.hc_compact_pages(None, None, 0, 0, 0, None, None, 0, None, None, 0, None) == B.HC_ERR_INVALID
