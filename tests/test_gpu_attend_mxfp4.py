"""Attention over a cache held in 4 bits, against 64 bits: the cases of the cache of elements, its values those that the
codes stand for."""
import math

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests import mxfp4_support as M
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu


class Case4(Case):
    """A Case whose pool holds 4-bit rows; `host` is what they stand for, `fill` the bytes that are not read."""

    def __init__(self, fill=0xff, **kw):
        super().__init__(**kw)
        self.host4 = [torch.stack([M.pack(t[l].double(), self.hk, t.shape[2] // self.hk, fill) for l in range(len(t))])
                      for t in self.host]
        self.read()

    def read(self):
        self.host = [M.unpack(t, self.hk, d).to(self.dt) for t, d in zip(self.host4, (self.d, self.dv))]

    def upload(self):
        self.dev = [t.cuda() for t in self.host4]
        self.pool = F.pool_of(self.dev, self.page)
        self.args = dict(kv_heads=self.hk, entry_tokens=self.entry, value_dim=self.dv, cache="mxfp4")
        self.on = dict(q=self.q.cuda(), table=self.table.cuda(), kv_len=self.kv_len.cuda(), q_start=self.q_start.cuda())
        return self


def check(kw=None, **case):
    c = Case4(**case).upload()
    c.check(**(kw or {}))
    c.close()


HEADS = [dict(hq=8, hk=2, d=64), dict(hq=8, hk=1, d=128), dict(hq=4, hk=4, d=128), dict(hq=6, hk=2, d=64),
         dict(hq=14, hk=2, d=128), dict(hq=20, hk=1, d=128), dict(hq=40, hk=2, d=64), dict(hq=32, hk=8, d=128),
         dict(hq=12, hk=12, d=64), dict(hq=9, hk=3, d=128), dict(hq=16, hk=1, d=576), dict(hq=3, hk=1, d=576),
         dict(hq=128, hk=1, d=576)]
NAMES = lambda h: f"{h['hq']}-{h['hk']}-{h['d']}"  # noqa: E731


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS, ids=NAMES)
def test_decode(heads, dtype):
    """One token per sequence, lengths around tile, page and split sizes."""
    check(dtype=dtype, kv=(1, 2, 15, 16, 17, 63, 64, 65, 129, 0, 300), q=(1,) * 11, page=24, **heads)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS[:-1], ids=NAMES)
def test_chunks(heads, dtype):
    """Chunks of unequal lengths behind cached prefixes of unequal lengths, and none."""
    check(dtype=dtype, kv=(70, 5, 33, 131, 64), q=(3, 5, 0, 40, 17), page=16, **heads)


@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("kv,q", [(257, 257), (129, 128), (300, 1), (511, 65), (1, 1), (200, 31), (1100, 9), (1500, 1)])
def test_one_sequence(d, kv, q):
    check(hq=4, hk=1 if d == 576 else 2, d=d, kv=(kv,), q=(q,), page=64, q_scale=3.0)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=7, sinks=1), dict(window=33, sinks=4), dict(window=16, sinks=40),
                                dict(window=64, sinks=100), dict(window=1000, sinks=3), dict(causal=False),
                                dict(scale=-0.3), dict(scale=0.0)])
@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("entry", [1, 16])
def test_masks(kw, d, entry):
    heads = dict(hq=6, hk=1 if d == 576 else 2, d=d)
    check(kw, kv=(150, 40, 3, 260), q=(1, 9, 3, 70), page=16, entry=entry, seed=3, **heads)
    check(kw, kv=(150, 40, 3, 260), q=(1, 1, 1, 1), page=16, entry=entry, seed=4, pad_rows=2, **heads)


@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("q", [(1, 1, 1), (5, 40, 70)])
def test_rows_that_see_nothing(d, q):
    """More new tokens than cached ones: the first rows stand before the sequence."""
    check(hq=4, hk=1 if d == 576 else 2, d=d, kv=(0, 30, 1), q=q, page=16)


@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("q", [(1, 1, 1), (3, 20, 10)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_hidden_rows_that_are_not_numbers(d, q, dtype):
    """What stands behind a sequence, before its window and after a row's position is NaN, or infinite in fp16."""
    c = Case4(hq=4, hk=1 if d == 576 else 2, d=d, kv=(90, 200, 70), q=q, page=16, seed=7, dtype=dtype)
    n = c.hk * c.d
    for s, kv in enumerate((90, 200, 70)):
        slot = F.slots_of(c.table[s].clamp(min=0), -(-kv // 16) * 16, 16)
        hidden = torch.cat([slot[:20], slot[kv:]])  # before the window of 30, and the page's rest
        for t in c.host4:
            t[1, hidden, n // 2:n // 2 + n // 32] = 255 if s != 1 else 250
    c.read()
    c.upload().check(window=30)
    c.close()


@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("q", [(1, 1), (6, 40)])
def test_visible_values_that_are_not_numbers(d, q):
    """A NaN block of values is NaN in its dims only, a NaN key makes the rows that see it NaN."""
    c = Case4(hq=4, hk=1 if d == 576 else 2, d=d, kv=(90, 150), q=q, page=16, seed=8)
    n = c.hk * c.d
    t = c.host4[-1]
    slot = F.slots_of(c.table[1], 150, 16)
    t[1, slot[10], n // 2] = 255
    c.read()
    c.upload()
    out, lse = c.run()
    torch.cuda.synchronize()
    w, wl, tol, tl = c.want()
    if d == 576:  # the key is NaN too
        rows = int(c.q_start[1])
        assert out[rows:].isnan().all() and lse[rows:].isnan().all()
        F.close(out[:rows], w[:rows], tol[:rows], "out")
    else:
        F.close(out, w, torch.nan_to_num(tol, 0.0), "out")
        F.close(lse, wl, tl, "lse")
    c.pool.sync()
    c.close()


def test_bad_entries_and_lengths_are_reported():
    for d in (64, 128, 576):
        for q in ((1, 1, 1), (4, 40, 3)):
            c = Case4(hq=4, hk=1 if d == 576 else 2, d=d, kv=(70, 90, 50), q=q, page=16)
            c.upload()
            c.on["table"][1, 2] = 10 ** 6  # (the oracle goes by the table as it was, those keys hidden)
            out, lse = c.run()
            with pytest.raises(B.HcError) as e:
                c.pool.sync()
            assert e.value.code == B.HC_ERR_DEVICE
            w, wl, tol, tl = c.want(hidden=[(1, k) for k in range(32, 48)])
            F.close(out, w, tol, "out")
            F.close(lse, wl, tl, "lse")
            c.on["kv_len"][2] = 1000
            out = torch.full_like(out, 9.0)
            c.run(out=out)
            with pytest.raises(B.HcError):
                c.pool.sync()
            at = int(c.q_start[2])
            assert out[at:].eq(9.0).all()
            F.close(out[:at], w[:at], tol[:at], "out")
            c.close()


@pytest.mark.parametrize("d", [64, 128, 576])
def test_many_sequences_and_mixes(d):
    heads = dict(hq=8, hk=1 if d == 576 else 2, d=d)
    g = torch.Generator().manual_seed(9)
    kv = torch.randint(0, 90, (300,), generator=g).tolist()
    check(kv=kv, q=(1,) * 300, page=16, **heads)
    check(kv=(700, 20, 300, 64, 65), q=(1, 20, 33, 1, 2), page=24, **heads)


@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_strides_and_streams(d, dtype):
    """Queries out of a fused projection, out between other rows, on a named stream, no lse."""
    c = Case4(hq=4, hk=1 if d == 576 else 2, d=d, kv=(90, 33), q=(1, 5), page=16, seed=2, dtype=dtype).upload()
    wide = torch.zeros((c.rows, 2, c.hq, d + 8), dtype=c.dt, device="cuda")
    wide[:, 1, :, :d] = c.on["q"]
    c.on["q"] = wide[:, 1, :, :d]
    out = torch.full((c.hq, c.rows, c.dv), 9.0, dtype=c.dt, device="cuda").transpose(0, 1)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(out=out, return_lse=False, stream=stream)
    stream.synchronize()
    w, _, tol, _ = c.want()
    F.close(out, w, tol, "out")
    c.pool.sync()
    c.close()


@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("q", [(1, 1), (20, 40)])
def test_captured(d, q):
    """One graph, replayed over other lengths, rows and queries; every replay like the eager call."""
    c = Case4(hq=8, hk=1 if d == 576 else 2, d=d, kv=(400, 300), q=q, page=16, seed=6).upload()
    out = torch.empty((c.rows, c.hq, c.dv), dtype=c.dt, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        _, lse = c.run(out=out)
    for kv in ((400, 300), (41, 300), (0, 50), (399, 64)):
        c.kv_len = torch.tensor(kv)
        c.on["kv_len"].copy_(c.kv_len)
        c.on["q"].neg_()
        graph.replay()
        torch.cuda.synchronize()
        again, lse2 = c.run()
        torch.cuda.synchronize()
        assert torch.equal(F.bits(again.cpu()), F.bits(out.cpu())) and torch.equal(lse, lse2)
        c.q = c.on["q"].cpu()
        c.compare(out, lse, c.want())
    c.pool.sync()
    del graph
    c.close()


def test_refusals():
    c = Case4(hq=4, hk=2, d=64, kv=(40,), q=(1,), page=16).upload()
    for kw, code in [(dict(cache="elements"), B.HC_ERR_INVALID), (dict(kv_heads=1), B.HC_ERR_INVALID),
                     (dict(scale=math.nan), B.HC_ERR_INVALID), (dict(window=4, causal=False), B.HC_ERR_INVALID),
                     (dict(out=c.on["q"]), B.HC_ERR_INVALID)]:
        args = dict(dict(kv_heads=2, cache="mxfp4", max_kv=40), **kw)
        with pytest.raises(B.HcError) as e:
            c.pool.attend(1, c.on["q"], c.on["table"], c.on["kv_len"], **args)
        assert e.value.code == code, e.value
    with pytest.raises(ValueError):
        c.pool.attend(1, c.on["q"], c.on["table"], c.on["kv_len"], kv_heads=2, cache="fp4")
    rows = c.dev[0][1].view(torch.bfloat16).flatten()[:256].view(1, 4, 64)
    with pytest.raises(B.HcError):
        c.pool.attend(1, c.on["q"], c.on["table"], c.on["kv_len"], kv_heads=2, cache="mxfp4", out=rows)
    c.pool.sync()
    c.close()
