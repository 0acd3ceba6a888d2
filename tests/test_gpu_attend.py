"""Attention over the device pool, against 64 bits."""
import ctypes
import math

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F

pytestmark = pytest.mark.gpu


def normal(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, dtype=torch.float64) * scale


class Case:
    """A pool of one or two sub-buffers, sequences in random places of it, packed queries."""

    def __init__(self, *, dtype="bf16", hq=8, hk=2, d=64, page=16, entry=None, kv=(40,), q=(1,), seed=0, layers=2,
                 layer=1, pad_rows=0, q_scale=1.0, extra_width=0):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.hq, self.hk, self.d = F.DTYPES[dtype], hq, hk, d
        self.dv = 512 if d == 576 else d
        self.page, self.entry, self.layer = page, page if entry is None else entry, layer
        self.kv, self.q_len = list(kv), list(q)
        used = [-(-n // page) for n in kv]
        pages = sum(used) + 3
        S = pages * page
        self.host = [normal(g, layers, S, hk * e).to(self.dt) for e in ([d] if d == 576 else [d, d])]
        width = max([-(-n // self.entry) for n in kv] + [1]) + extra_width
        place = torch.randperm(S // self.entry, generator=g)
        table = torch.full((len(kv), width), -1, dtype=torch.int64)
        at = 0
        for s, n in enumerate(kv):
            m = -(-n // self.entry)
            table[s, :m] = place[at:at + m]
            at += m
        self.table = table
        self.q_start = torch.tensor([0] + self.q_len).cumsum(0)
        self.rows = int(self.q_start[-1]) + pad_rows
        self.q = normal(g, self.rows, hq, d, scale=q_scale).to(self.dt)
        self.kv_len = torch.tensor(self.kv, dtype=torch.int64)

    def upload(self):
        self.dev = [t.cuda() for t in self.host]
        self.pool = F.pool_of(self.dev, self.page)
        self.args = dict(kv_heads=self.hk, entry_tokens=self.entry, value_dim=self.dv)
        self.on = dict(q=self.q.cuda(), table=self.table.cuda(), kv_len=self.kv_len.cuda(),
                       q_start=self.q_start.cuda())
        return self

    def run(self, *, out=None, return_lse=True, **kw):
        if out is None:
            out = torch.full((self.rows, self.hq, self.dv), 9.0, dtype=self.dt, device="cuda")
        kw = dict(dict(max_q=max(self.q_len, default=0), max_kv=max(self.kv, default=0)), **kw)
        return self.pool.attend(self.layer, self.on["q"], self.on["table"], self.on["kv_len"],
                                q_start=self.on["q_start"], out=out, return_lse=return_lse, **self.args, **kw)

    def want(self, hidden=(), **kw):
        kw = {k: v for k, v in kw.items() if k in ("causal", "window", "sinks", "scale")}
        return F.attend(self.q, self.host[0][self.layer], None if self.d == 576 else self.host[1][self.layer],
                        self.table, self.kv_len, self.q_start, kv_heads=self.hk, entry=self.entry,
                        value_dim=self.dv, hidden=hidden, **kw)

    def check(self, **kw):
        out, lse = self.run(**kw)
        torch.cuda.synchronize()
        self.pool.sync()
        self.compare(out, lse, self.want(**kw))

    def compare(self, out, lse, want):
        w, wl, tol, tol_l = want
        n = int(self.q_start[-1])
        F.close(out[:n], w[:n], tol[:n], "out")
        F.close(lse[:n], wl[:n], tol_l[:n], "lse")
        if self.rows > n:
            assert out[n:].eq(9.0).all()

    def close(self):
        self.pool.close()


def check(kw=None, **case):
    c = Case(**case).upload()
    c.check(**(kw or {}))
    c.close()


HEADS = [dict(hq=8, hk=2, d=64), dict(hq=8, hk=1, d=128), dict(hq=4, hk=4, d=128), dict(hq=6, hk=2, d=64),
         dict(hq=14, hk=2, d=128), dict(hq=20, hk=1, d=128), dict(hq=40, hk=2, d=64), dict(hq=16, hk=1, d=576),
         dict(hq=3, hk=1, d=576), dict(hq=128, hk=1, d=576)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: f"{h['hq']}-{h['hk']}-{h['d']}")
def test_decode(heads, dtype):
    """One token per sequence, lengths around tile, page and split sizes."""
    check(dtype=dtype, kv=(1, 2, 15, 16, 17, 63, 64, 65, 129, 0, 300), q=(1,) * 11, page=24, **heads)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", HEADS[:-1], ids=lambda h: f"{h['hq']}-{h['hk']}-{h['d']}")
def test_chunks(heads, dtype):
    """Chunks of unequal lengths behind cached prefixes of unequal lengths, and none."""
    check(dtype=dtype, kv=(70, 5, 33, 131, 64), q=(3, 5, 0, 40, 17), page=16, **heads)


@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("kv,q", [(257, 257), (129, 128), (300, 1), (511, 65), (1, 1), (200, 31), (1100, 9)])
def test_one_sequence(d, kv, q):
    check(hq=4, hk=1 if d == 576 else 2, d=d, kv=(kv,), q=(q,), page=64, q_scale=3.0)


@pytest.mark.parametrize("kw", [dict(window=1), dict(window=7, sinks=1), dict(window=33, sinks=4),
                                dict(window=16, sinks=40), dict(window=64, sinks=100), dict(window=1000, sinks=3),
                                dict(window=100, sinks=1 << 40)])
@pytest.mark.parametrize("d", [64, 128, 576])
def test_windows_and_sinks(kw, d):
    check(kw, hq=4, hk=1 if d == 576 else 2, d=d, kv=(300, 40, 7, 129, 90), q=(70, 40, 1, 1, 2), page=16, entry=1)


@pytest.mark.parametrize("kw", [dict(), dict(window=20, sinks=3)])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1), (576, 4, 1)])
def test_a_few_tokens_a_sequence(d, hq, hk, kw):
    """Several new tokens in the decoding kernels' row tiles, splits among them."""
    check(kw, hq=hq, hk=hk, d=d, kv=(300, 40, 1000, 2, 700), q=(2, 4, 3, 1, 4), page=16)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("d,q", [(64, (1, 1)), (64, (30, 33)), (128, (40, 3)), (576, (1, 1)), (576, (40, 9))])
def test_any_scale(d, q, scale):
    check(dict(scale=scale), hq=4, hk=1 if d == 576 else 2, d=d, kv=(150, 70), q=q, page=16)


@pytest.mark.parametrize("d,hq,hk", [(64, 2, 1), (576, 2, 1)])
@pytest.mark.parametrize("seqs,q", [(4, 1), (5, 1), (256, 1), (257, 1), (700, 1), (300, 40)])
def test_many_sequences(d, hq, hk, seqs, q):
    """The list of work over one, several and very many sequences, empty ones among them."""
    if q > 1 and d == 576:
        q = 20
    g = torch.Generator().manual_seed(seqs)
    kv = torch.randint(0, 40, (seqs,), generator=g).tolist()
    kv[seqs // 2] = 1500
    qs = [1] * seqs if q == 1 else [q if i % 97 == 5 else i % 2 for i in range(seqs)]
    qs = [min(a, max(b, 1)) for a, b in zip(qs, kv)]
    check(hq=hq, hk=hk, d=d, kv=kv, q=qs, page=8)


def test_a_chunk_beside_long_decoding_sequences():
    """One call of a chunk that fills the GPU and decoding rows of long sequences, which are split:
    every decoding row and some of the chunk's against 64 bits, the lengths shorter than their bound."""
    c = Case(hq=32, hk=8, d=64, kv=(17000, 2100, 20000, 3), q=(1, 2050, 1, 1), page=64).upload()
    out, lse = c.run(max_q=2050, max_kv=20032)
    torch.cuda.synchronize()
    c.pool.sync()
    for row, s, p in [(0, 0, 16999), (1, 1, 50), (7, 1, 56), (130, 1, 179), (2050, 1, 2099), (2051, 2, 19999), (2052, 3, 2)]:
        w, wl, tol, tol_l = F.attend(c.q[row:row + 1], c.host[0][1], c.host[1][1], c.table[s:s + 1], [p + 1], [0, 1],
                                     kv_heads=8, entry=64)
        F.close(out[row:row + 1], w, tol, f"row {row}")
        F.close(lse[row:row + 1], wl, tol_l, f"lse {row}")
    c.close()


@pytest.mark.parametrize("d", [64, 128, 576])
def test_without_causality(d):
    check(dict(causal=False), hq=4, hk=1 if d == 576 else 2, d=d, kv=(150, 20, 3), q=(20, 20, 9), page=16)


@pytest.mark.parametrize("d", [64, 128, 576])
def test_rows_that_see_nothing(d):
    """More new tokens than cached ones, no cached token at all: zeros and -infinity."""
    c = Case(hq=4, hk=1 if d == 576 else 2, d=d, kv=(3, 0, 10, 0), q=(8, 2, 1, 1), pad_rows=5).upload()
    out, lse = c.run()
    c.compare(out, lse, c.want())
    assert out[:5].eq(0).all() and lse[:5].eq(-math.inf).all() and out[8:10].eq(0).all()
    c.close()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("q", [(1, 1), (6, 50)])
def test_what_is_not_seen_does_not_matter(q, d, bad):
    """Infinities and NaN in every row of the pool that no query sees, and in keys and values
    that later queries of the same tile see."""
    c = Case(hq=4, hk=1 if d == 576 else 2, d=d, kv=(37, 90), q=q, page=16)
    used = torch.zeros(c.host[0].shape[1], dtype=torch.bool)
    for s, n in enumerate(c.kv):
        used[F.slots_of(c.table[s], n, c.entry)] = True
    for t in c.host:
        t[:, ~used] = bad
    if q[1] > 1:  # the newest token of the second sequence: its own last row sees it alone
        for t in c.host:
            t[c.layer, F.slots_of(c.table[1], 90, c.entry)[-1]] = bad
    c.upload()
    out, lse = c.run(window=30, sinks=2)
    torch.cuda.synchronize()
    w, wl, tol, tol_l = c.want(window=30, sinks=2)
    n = int(c.q_start[-1]) - (1 if q[1] > 1 else 0)
    F.close(out[:n], w[:n], tol[:n], "out")
    F.close(lse[:n], wl[:n], tol_l[:n], "lse")
    assert out[:n].isfinite().all()
    if q[1] > 1 and not (bad == -math.inf):
        assert not out[n].isfinite().all()
    c.close()


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_seen_show(d):
    """An infinite value that a row sees is in its output; the other heads and rows stay finite."""
    c = Case(hq=2, hk=2, d=d, kv=(50,), q=(20,), page=16)
    where = F.slots_of(c.table[0], 50, c.entry)[40]
    c.host[1][c.layer, where, 5] = math.inf  # one element of KV head 0
    c.upload()
    out, lse = c.run()
    torch.cuda.synchronize()
    first = 50 - 20
    for r in range(20):
        if first + r < 40:
            assert out[r].isfinite().all()
        else:
            assert out[r, 0, 5] == math.inf and out[r, 1].isfinite().all()
    c.close()


def test_large_scores_and_lowest_values():
    """Scores of thousands, and keys of the type's lowest value."""
    c = Case(hq=4, hk=2, d=128, kv=(100, 3), q=(7, 1), q_scale=200.0)
    c.host[0][c.layer, F.slots_of(c.table[0], 100, c.entry)[50]] = torch.finfo(torch.bfloat16).min / 2 ** 20
    c.upload().check()
    c.close()


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (16, 1, 576)])
def test_strides_scale_and_views(hq, hk, d):
    """q a view of a fused projection, out a transposed view, a wider table, rows behind the batch."""
    c = Case(hq=hq, hk=hk, d=d, kv=(90, 31), q=(11, 1), pad_rows=3, extra_width=5).upload()
    fused = torch.zeros((c.rows, hq + 4, d), dtype=c.dt, device="cuda")
    fused[:, 2:2 + hq] = c.q.cuda()
    c.on["q"] = fused[:, 2:2 + hq]
    big = torch.full((c.table.shape[0], c.table.shape[1] + 9), 1 << 50, dtype=torch.int64, device="cuda")
    big[:, :c.table.shape[1]] = c.table.cuda()
    c.on["table"] = big[:, :c.table.shape[1]]
    out = torch.full((hq, c.rows, c.dv), 9.0, dtype=c.dt, device="cuda").transpose(0, 1)
    got, lse = c.run(out=out, scale=0.03)
    torch.cuda.synchronize()
    c.pool.sync()
    assert got is out
    c.compare(out, lse, c.want(scale=0.03))
    c.close()


def test_bad_entries_and_lengths_are_reported():
    c = Case(hq=4, hk=2, d=64, kv=(60, 33, 20, 50), q=(2, 1, 3, 1), page=16).upload()
    c.on["table"][0, 1] = 1 << 45          # hides tokens 16..31 of sequence 0
    c.on["kv_len"][1] = 1 << 40            # skipped
    c.on["kv_len"][2] = -1                 # skipped
    out, lse = c.run()
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="index out of range; a sequence's lengths out of bounds"):
        c.pool.sync()
    c.pool.sync()
    w, wl, tol, tol_l = c.want(hidden=[(0, j) for j in range(16, 32)])
    for rows in (slice(0, 2), slice(6, 7)):
        F.close(out[rows], w[rows], tol[rows], "out")
        F.close(lse[rows], wl[rows], tol_l[rows], "lse")
    assert out[2:6].eq(9.0).all()
    # q_start that goes back or past the queries
    c.on["kv_len"].copy_(c.kv_len)
    c.on["table"].copy_(c.table)
    c.on["q_start"].copy_(torch.tensor([0, 2, 1, 1 << 40, 7]))
    out, lse = c.run()
    torch.cuda.synchronize()
    with pytest.raises(B.HcError, match="lengths out of bounds"):
        c.pool.sync()
    assert out[2:].eq(9.0).all()
    # more rows, or tokens, than the call was told of
    c.on["q_start"].copy_(c.q_start)
    out, _ = c.run(max_q=2)
    assert out[3:6].eq(9.0).all() and not out[:2].eq(9.0).any()
    out, _ = c.run(max_kv=50)
    assert out[:2].eq(9.0).all() and not out[2:].eq(9.0).all()
    with pytest.raises(B.HcError):
        c.pool.sync()
    c.close()


def test_refusals():
    c = Case(hq=4, hk=2, d=64, kv=(20,), q=(2,)).upload()

    def refuse(code, **kw):
        with pytest.raises(B.HcError) as e:
            c.run(**kw)
        assert e.value.code == code, e.value

    refuse(B.HC_ERR_INVALID, scale=math.nan)
    refuse(B.HC_ERR_INVALID, window=-1)
    refuse(B.HC_ERR_INVALID, window=4, causal=False)
    refuse(B.HC_ERR_INVALID, max_kv=1000)                       # more than a table row holds
    refuse(B.HC_ERR_INVALID, out=c.on["q"])
    c.args["entry_tokens"] = 3
    refuse(B.HC_ERR_INVALID)
    c.args["entry_tokens"] = c.entry
    c.args["kv_heads"] = 3
    refuse(B.HC_ERR_INVALID)
    c.args["kv_heads"] = 4                                     # rows of another size
    refuse(B.HC_ERR_INVALID)
    c.args["kv_heads"] = 2
    c.layer = 2
    refuse(B.HC_ERR_INVALID)
    c.layer = 1
    c.args["value_dim"] = 32
    refuse(B.HC_ERR_UNSUPPORTED, out=torch.empty((2, 4, 32), dtype=c.dt, device="cuda"))
    c.args["value_dim"] = 64
    wide = torch.zeros((2, 4, 100), dtype=c.dt, device="cuda")
    refuse(B.HC_ERR_UNSUPPORTED, out=wide[..., :64])
    q = c.on["q"]
    c.on["q"] = q.float()
    with pytest.raises(TypeError):
        c.run()
    c.on["q"] = q
    c.on["table"] = c.on["table"].int()
    with pytest.raises(TypeError):
        c.run()
    c.on["table"] = c.table.cuda()
    out, _ = c.run(return_lse=False)
    assert _ is None
    d = B.hc_attend_desc()
    assert B.lib.hc_attend(c.pool.handle, ctypes.byref(d), None) == B.HC_ERR_INVALID
    c.close()


@pytest.mark.parametrize("q,kv", [((1, 1, 1), (900, 5, 333)), ((40, 3, 1), (500, 3, 777))])
@pytest.mark.parametrize("d", [64, 576])
def test_captured_and_replayed(q, kv, d):
    """A captured call replayed on new contents, beside eager work, each replay against eager."""
    c = Case(hq=8, hk=1 if d == 576 else 2, d=d, kv=kv, q=q, page=16).upload()
    out = torch.zeros((c.rows, c.hq, c.dv), dtype=c.dt, device="cuda")
    c.run(out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = c.run(out=out)
    for k in range(3):
        c.on["q"].copy_(torch.randn_like(c.on["q"]))
        c.on["kv_len"][0] = kv[0] - 7 * k
        eager, eager_lse = c.run()
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(F.bits(out), F.bits(eager)) and torch.equal(lse, eager_lse), k
    c.pool.sync()
    del graph
    c.close()


def test_two_streams_at_once():
    """Calls on two streams, each with its own workspace, agree with one after the other."""
    cs = [Case(hq=8, hk=2, d=128, kv=(3000, 1500), q=(1, 1), page=16, seed=s).upload() for s in range(2)]
    want = [c.run() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[] for _ in cs]
    for _ in range(8):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                got[i].append(c.run())
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(F.bits(out), F.bits(want[i][0])) and torch.equal(lse, want[i][1])
    # a named stream
    s = torch.cuda.Stream()
    out, lse = cs[0].run(stream=s)
    s.synchronize()
    assert torch.equal(F.bits(out), F.bits(want[0][0]))
    for c in cs:
        c.close()


def test_same_result_every_time():
    c = Case(hq=16, hk=2, d=128, kv=(2000, 70, 900), q=(33, 70, 1), page=16).upload()
    out, lse = c.run()
    for _ in range(4):
        o, l = c.run()
        assert torch.equal(F.bits(o), F.bits(out)) and torch.equal(l, lse)
    c.close()


@pytest.mark.parametrize("m", [5, 50])
@pytest.mark.parametrize("hk,d", [(8, 128), (1, 576)])
@pytest.mark.parametrize("entry", [1, 64])
def test_rows_past_two_gigabytes(entry, hk, d, m):
    """A pool whose rows lie past 2^32 bytes of a layer, and past 2^31 elements."""
    page, hq = 64, 2 * hk
    S = (5 << 30) // (hk * d * 2) // page * page
    subs = 1 if d == 576 else 2
    dev = [torch.zeros((1, S, hk * d), dtype=torch.bfloat16, device="cuda") for _ in range(subs)]
    pool = F.pool_of(dev, page)
    g = torch.Generator().manual_seed(3)
    n = 200
    slots = S - 1 - torch.arange(n) if entry == 1 else torch.arange(n) + S - 4 * page
    rows = [normal(g, n, hk * d).to(torch.bfloat16) for _ in range(subs)]
    for t, r in zip(dev, rows):
        t[0][slots.cuda()] = r.cuda()
    table = slots[None] if entry == 1 else torch.arange(4)[None] + S // page - 4
    q = normal(g, m, hq, d).to(torch.bfloat16)
    dv = 512 if d == 576 else d
    out, lse = pool.attend(0, q.cuda(), table.cuda(), torch.tensor([n]).cuda(), kv_heads=hk, value_dim=dv,
                           q_start=torch.tensor([0, m]).cuda(), entry_tokens=entry, return_lse=True)
    w, wl, tol, tol_l = F.attend(q, rows[0], None if subs == 1 else rows[1], torch.arange(n)[None], [n], [0, m],
                                 kv_heads=hk, entry=1, value_dim=dv)
    F.close(out, w, tol, "out")
    F.close(lse, wl, tol_l, "lse")
    pool.sync()
    pool.close()
