"""Attention over a 4-bit cache where sequences are split and joined, where calls have fewer places than items, where a
latent cache is converted first, and what workspaces hold."""
import ctypes

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests.test_gpu_attend_mxfp4 import Case4, check

pytestmark = pytest.mark.gpu

FEW = [dict(hq=4, hk=1, d=64), dict(hq=4, hk=2, d=128), dict(hq=8, hk=4, d=128), dict(hq=8, hk=8, d=64), dict(hq=4, hk=1, d=576)]
NAMES = lambda h: f"{h['hq']}-{h['hk']}-{h['d']}"  # noqa: E731


@pytest.mark.parametrize("heads", FEW, ids=NAMES)
def test_one_long_sequence(heads):
    """More splits than a wave has lanes, and the fewest."""
    check(kv=(9000,), q=(1,), page=64, **heads)
    check(kv=(140,), q=(2,), page=64, **heads)
    check(dict(window=700, sinks=5), kv=(3000,), q=(1,), page=16, entry=1, dtype="fp16", **heads)


@pytest.mark.parametrize("heads", FEW, ids=NAMES)
def test_many_rows_joined_by_waves(heads):
    """More rows than a workgroup each joins, tiles of a few and of more tokens, beside sequences that are not split."""
    g = torch.Generator().manual_seed(1)
    kv = torch.randint(0, 500, (140,), generator=g).tolist()
    check(kv=kv, q=(1,) * 140, page=16, **heads)
    check(kv=(900, 30, 1200, 64), q=(5, 2, 7, 1), page=24, **heads)


@pytest.mark.parametrize("heads", [dict(hq=2, hk=1, d=64), dict(hq=2, hk=1, d=576)], ids=NAMES)
def test_more_items_than_places(heads):
    """Thousands of short sequences beside one that is split."""
    n = 2300
    kv = [3] * n
    kv[n // 2] = 2100
    check(kv=kv, q=(1,) * n, page=8, **heads)


@pytest.mark.parametrize("heads", [dict(hq=4, hk=1, d=64), dict(hq=6, hk=2, d=128), dict(hq=2, hk=1, d=576)], ids=NAMES)
def test_chunks_beside_decoding_rows(heads):
    """Many rows of one sequence, one of others, split and not."""
    check(kv=(700, 400, 90, 650), q=(120, 1, 1, 33), page=16, **heads)


LATENT = dict(hq=16, hk=1, d=576)  # 512 rows of a sequence are 32 of its tokens


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kw", [dict(), dict(window=50, sinks=3), dict(causal=False), dict(scale=-0.2)])
def test_latent_chunks_converted_first(kw, dtype):
    check(kw, kv=(90, 40, 0, 3), q=(35, 1, 0, 3), page=16, dtype=dtype, seed=1, pad_rows=1, **LATENT)
    check(kw, kv=(70, 33), q=(34, 33), page=24, entry=1, dtype=dtype, seed=2, **LATENT)


def test_latent_chunks_with_bad_entries_and_lengths():
    c = Case4(kv=(90, 80, 50), q=(33, 34, 3), page=16, **LATENT).upload()
    c.on["table"][1, 2] = -3
    out, lse = c.run()
    with pytest.raises(B.HcError) as e:
        c.pool.sync()
    width = c.table.shape[1]
    assert e.value.code == B.HC_ERR_DEVICE and str(width + 2) in str(e.value)
    w, wl, tol, tl = c.want(hidden=[(1, k) for k in range(32, 48)])
    F.close(out, w, tol, "out")
    F.close(lse, wl, tl, "lse")
    c.on["table"][1, 2] = c.table[1, 2]
    c.on["kv_len"][0] = 1000
    out = torch.full_like(out, 9.0)
    c.run(out=out)
    with pytest.raises(B.HcError) as e:
        c.pool.sync()
    assert e.value.code == B.HC_ERR_DEVICE and "0" in str(e.value)
    w, _, tol, _ = c.want()
    assert out[:33].eq(9.0).all()
    F.close(out[33:], w[33:], tol[33:], "out")
    c.pool.sync()
    c.close()


def test_latent_chunks_beside_rows_that_are_not_numbers():
    """Behind the sequence and before the window NaN; a visible NaN key makes its rows NaN."""
    c = Case4(kv=(120, 70), q=(33, 32), page=16, seed=3, **LATENT)
    slot = F.slots_of(c.table[0], 128, 16)
    c.host4[0][1, slot[:40], 288:306] = 255
    c.host4[0][1, slot[120:], 288:306] = 255
    other = F.slots_of(c.table[1], 70, 16)
    c.host4[0][1, other[60], 288] = 255
    c.read()
    c.upload()
    out, lse = c.run(window=30)
    torch.cuda.synchronize()
    w, wl, tol, tl = c.want(window=30)
    F.close(out, w, torch.nan_to_num(tol), "out")
    F.close(lse, wl, torch.nan_to_num(tl), "lse")
    assert out[:33].isfinite().all() and out[33 + 22:].isnan().all()
    c.pool.sync()
    c.close()


def test_a_latent_chunk_captured():
    c = Case4(kv=(100, 60), q=(33, 34), page=16, seed=5, **LATENT).upload()
    out = torch.empty((c.rows, c.hq, c.dv), dtype=c.dt, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        _, lse = c.run(out=out)
    for kv in ((100, 60), (33, 40), (0, 60)):
        c.kv_len = torch.tensor(kv)
        c.on["kv_len"].copy_(c.kv_len)
        graph.replay()
        torch.cuda.synchronize()
        again, lse2 = c.run()
        torch.cuda.synchronize()
        assert torch.equal(F.bits(again.cpu()), F.bits(out.cpu())) and torch.equal(lse, lse2)
        c.compare(out, lse, c.want())
    c.pool.sync()
    del graph
    c.close()


@pytest.mark.parametrize("heads,kv,q", [
    (dict(hq=4, hk=1, d=64), (3000,), (1,)), (dict(hq=8, hk=4, d=128), (900, 2000), (2, 1)),
    (dict(hq=4, hk=1, d=576), (2000, 300), (1, 3)), (dict(hq=6, hk=2, d=128), (900, 200), (60, 1)),
    (dict(hq=4, hk=1, d=576), (900, 200), (30, 1)), (dict(hq=16, hk=1, d=576), (300, 60), (34, 1))],
    ids=lambda x: NAMES(x) if isinstance(x, dict) else str(x))
def test_ends_of_workspaces(heads, kv, q):
    """A workspace of exactly the bytes asked for: nothing around it is written, less is refused, what it held does not
    matter."""
    c = Case4(kv=kv, q=q, page=16, **heads).upload()
    need = ctypes.c_int64()
    d = B.hc_attend_desc(layer=1, dtype=B.HC_BF16, q_heads=c.hq, kv_heads=c.hk, head_dim=c.d, value_dim=c.dv,
                         value_in_key=int(c.d != c.dv), causal=1, entry_tokens=16, scale=1.0, num_seqs=len(kv), q_rows=c.rows,
                         max_q=max(q), max_kv=max(kv), table_width=c.table.shape[1], table_stride=c.table.shape[1])
    assert B.lib.hc_attend_mxfp4_workspace_bytes(c.pool.handle, ctypes.byref(d), ctypes.byref(need)) == B.HC_OK
    n = need.value
    assert n > 0
    raw = torch.full((n + 8192,), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = c.run(workspace=raw[4096:4096 + n])
    torch.cuda.synchronize()
    c.compare(out, lse, c.want())
    assert raw[:4096].eq(0xff).all() and raw[4096 + n:].eq(0xff).all()
    with pytest.raises(B.HcError) as e:
        c.run(workspace=raw[4096:4096 + n - 16])
    assert e.value.code == B.HC_ERR_INVALID
    c.pool.sync()
    c.close()


def test_two_calls_at_once():
    """Two streams with workspaces of their own."""
    a = Case4(hq=8, hk=4, d=128, kv=(2500, 700), q=(1, 1), page=16, seed=1).upload()
    b = Case4(hq=4, hk=1, d=576, kv=(1500, 900), q=(1, 2), page=16, seed=2).upload()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(4):
        for c, s, o in zip((a, b), streams, outs):
            o.append(c.run(stream=s))
    torch.cuda.synchronize()
    for c, o in zip((a, b), outs):
        want = c.want()
        for x in o:
            c.compare(*x, want)
        c.pool.sync()
        c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_latent_chunks_whose_bound_is_too_far_to_convert(dtype):
    """The same rows under a bound of tokens whose elements would be too many bytes."""
    c = Case4(kv=(90, 40), q=(35, 1), page=16, dtype=dtype, extra_width=20000, **LATENT).upload()
    c.check(max_kv=300000)
    near, far = c.run(), c.run(max_kv=300000)
    torch.cuda.synchronize()
    F.close(far[0], near[0].double().cpu(), 2 * c.want()[2], "out")
    c.pool.sync()
    c.close()


@pytest.mark.parametrize("heads", [dict(hq=16, hk=8, d=128), dict(hq=16, hk=8, d=64), dict(hq=12, hk=6, d=128),
                                   dict(hq=6, hk=3, d=64), dict(hq=16, hk=1, d=576)], ids=NAMES)
def test_sequences_that_are_named_twice(heads):
    """A q_start that goes back between sequences is reported; the list of work is then longer than the launch, which ends
    inside a tile, and what is left of it stays inside the workspace."""
    n = 20011
    c = Case4(kv=(n,), q=(1,), page=64, **heads).upload()
    seqs = 33
    c.on["q_start"] = (torch.arange(seqs + 1) % 2).cuda()
    c.on["kv_len"] = torch.full((seqs,), n).cuda()
    c.on["table"] = c.table.expand(seqs, -1).contiguous().cuda()
    need = ctypes.c_int64()
    width = c.table.shape[1]
    d = B.hc_attend_desc(layer=1, dtype=B.HC_BF16, q_heads=c.hq, kv_heads=c.hk, head_dim=c.d, value_dim=c.dv,
                         value_in_key=int(c.d != c.dv), causal=1, entry_tokens=64, scale=1.0, num_seqs=seqs, q_rows=1,
                         max_q=1, max_kv=n, table_width=width, table_stride=width)
    assert B.lib.hc_attend_mxfp4_workspace_bytes(c.pool.handle, ctypes.byref(d), ctypes.byref(need)) == B.HC_OK
    raw = torch.full((need.value + (1 << 24),), 0xff, dtype=torch.uint8, device="cuda")
    mid = raw[1 << 23:(1 << 23) + need.value]
    out, _ = c.run(workspace=mid, max_q=1, max_kv=n)
    with pytest.raises(B.HcError, match="lengths out of bounds; first flagged list position 1"):
        c.pool.sync()
    assert raw[:1 << 23].eq(0xff).all() and raw[(1 << 23) + need.value:].eq(0xff).all()
    assert out.isfinite().all()
    c.close()
