"""Attention whose sequences are split over workgroups, some or all: what a call needs as workspace, calls of many
unsplit rows beside split ones, lists of every mix of lengths, and the latent kernel of 17 to 32 rows."""
import ctypes
import math

import pytest
import torch

from host_device_page_amd import binding as B
from tests import forward_support as F
from tests.test_gpu_attend import Case, check

pytestmark = pytest.mark.gpu


def slot_bytes(d):
    """A partial result and what the joining launch knows of it, of the kernel of many rows."""
    return 4 * 64 * 514 + 32 if d == 576 else 4 * 128 * (d + 2) + 32


@pytest.mark.parametrize("rows,seqs,hq,hk,d", [(8192, 2, 32, 8, 128), (65536, 2, 32, 8, 128), (32768, 4, 128, 8, 128),
                                               (16384, 2, 64, 64, 64), (8192, 64, 128, 1, 576), (1 << 20, 999, 128, 1, 576)])
def test_the_workspace_does_not_grow_with_the_call(rows, seqs, hq, hk, d):
    """However many rows, splits are less than twice what runs at once."""
    dev = [torch.zeros((1, 64, hk * d), dtype=torch.bfloat16, device="cuda") for _ in range(1 if d == 576 else 2)]
    pool = F.pool_of(dev, 64)
    a = B.hc_attend_desc(layer=0, dtype=B.HC_BF16, q_heads=hq, kv_heads=hk, head_dim=d, value_dim=512 if d == 576 else d,
                         value_in_key=d == 576, causal=1, entry_tokens=64, scale=1.0, num_seqs=seqs, q_rows=rows,
                         max_q=rows, max_kv=1 << 17, table_width=1 << 11, table_stride=1 << 11)
    need = ctypes.c_int64()
    assert B.lib.hc_attend_workspace_bytes(pool.handle, ctypes.byref(a), ctypes.byref(need)) == B.HC_OK
    at_once = torch.cuda.get_device_properties(0).multi_processor_count * (1 if d == 576 else 2)
    assert 0 <= need.value <= 2 * at_once * slot_bytes(d) + 32
    pool.close()


def with_canary(c, **kw):
    """c.run with a workspace of exactly what it needs between bytes that have to stay."""
    need = ctypes.c_int64()
    hk, dv = c.hk, c.dv
    a = B.hc_attend_desc(layer=c.layer, dtype=B.HC_BF16 if c.dt == torch.bfloat16 else B.HC_F16, q_heads=c.hq, kv_heads=hk,
                         head_dim=c.d, value_dim=dv, value_in_key=dv != c.d, causal=1, entry_tokens=c.entry, scale=1.0,
                         num_seqs=len(c.on["kv_len"]), q_rows=c.rows, max_q=kw["max_q"], max_kv=kw["max_kv"],
                         table_width=c.on["table"].shape[1], table_stride=c.on["table"].stride(0))
    assert B.lib.hc_attend_workspace_bytes(c.pool.handle, ctypes.byref(a), ctypes.byref(need)) == B.HC_OK
    assert need.value > 0
    buf = torch.full((need.value + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = c.run(workspace=buf[4096:4096 + need.value], **kw)
    torch.cuda.synchronize()
    assert buf[:4096].eq(0xA5).all() and buf[4096 + need.value:].eq(0xA5).all()
    return out, lse


def rows_against_64_bits(c, out, lse, rows, heads=slice(None)):
    """Some rows of a causal call: (row, sequence, position), of some heads of a KV head's first."""
    for row, s, p in rows:
        w, wl, tol, tol_l = F.attend(c.q[row:row + 1, heads], c.host[0][1], None if c.d == 576 else c.host[1][1],
                                     c.table[s:s + 1], [p + 1], [0, 1], kv_heads=c.hk, entry=c.entry, value_dim=c.dv)
        F.close(out[row:row + 1, heads], w, tol, f"row {row}")
        F.close(lse[row:row + 1, heads], wl, tol_l, f"lse {row}")


@pytest.mark.parametrize("max_kv", [16384, 17408])
def test_a_chunk_beside_long_decoding_sequences_128(max_kv):
    """Heads of 128 on both sides of the length from which a call that fills the GPU is split."""
    long = max_kv - 300
    c = Case(hq=32, hk=8, d=128, kv=(long, 2100, long - 1000, 3), q=(1, 2050, 1, 1), page=64).upload()
    kw = dict(max_q=2050, max_kv=max_kv)
    c.on["table"] = torch.nn.functional.pad(c.table, (0, max_kv // 64 + 1 - c.table.shape[1]), value=-1).cuda()
    out, lse = with_canary(c, **kw) if max_kv > 16384 else c.run(**kw)
    torch.cuda.synchronize()
    c.pool.sync()
    rows_against_64_bits(c, out, lse, [(0, 0, long - 1), (1, 1, 50), (130, 1, 179), (2050, 1, 2099),
                                       (2051, 2, long - 1001), (2052, 3, 2)])
    c.close()


@pytest.mark.parametrize("max_kv", [16384, 17408])
@pytest.mark.parametrize("chunk", [20, 200])
def test_a_latent_chunk_beside_long_decoding_sequences(chunk, max_kv):
    """128 heads of a latent cache, row tiles that fill the GPU and that do not."""
    long = max_kv - 300
    c = Case(hq=128, hk=1, d=576, kv=(long, 400, 5), q=(1, chunk, 1), page=64).upload()
    kw = dict(max_q=chunk, max_kv=max_kv)
    c.on["table"] = torch.nn.functional.pad(c.table, (0, max_kv // 64 + 1 - c.table.shape[1]), value=-1).cuda()
    out, lse = with_canary(c, **kw) if max_kv > 16384 or chunk == 20 else c.run(**kw)
    torch.cuda.synchronize()
    c.pool.sync()
    rows = [(0, 0, long - 1), (1, 1, 400 - chunk), (chunk, 1, 399), (chunk + 1, 2, 4)]
    rows_against_64_bits(c, out, lse, rows, slice(0, 3))
    rows_against_64_bits(c, out, lse, rows, slice(125, 128))
    c.close()


@pytest.mark.parametrize("hq,hk,d", [(2, 1, 64), (3, 1, 128), (2, 1, 576), (16, 8, 64), (8, 8, 128)])
@pytest.mark.parametrize("seqs", [2, 5, 90, 600])
@pytest.mark.parametrize("many", [False, True])
def test_every_mix_of_lengths(hq, hk, d, seqs, many):
    """Lengths spread over their logarithm: split, unsplit and empty sequences in any order; many: some have
    more rows than a decoding tile."""
    if seqs == 600 and (many or hk == 8):
        seqs = 260
    g = torch.Generator().manual_seed(seqs + d)
    kv = torch.exp(torch.rand(seqs, generator=g) * math.log(4000)).long().tolist()
    kv[seqs // 2] = 0
    kv[-1] = 4000
    q = [35 if many and i % 23 == 1 else 1 for i in range(seqs)]
    c = Case(hq=hq, hk=hk, d=d, kv=kv, q=q, page=16).upload()
    out, lse = with_canary(c, max_q=max(q), max_kv=4000)
    c.pool.sync()
    c.compare(out, lse, c.want())
    c.close()


@pytest.mark.parametrize("hq,hk,d,pad", [(8, 8, 64, 10000), (8, 8, 128, 10000), (2, 1, 576, 7000)])
@pytest.mark.parametrize("seqs", [1, 3, 6])
def test_a_few_sequences_in_front_of_many_unused_rows(hq, hk, d, pad, seqs):
    """A padded batch whose row tiles, by the host's count, are more than there are places for partial results."""
    kv = [3000, 5, 0, 700, 64, 2000][:seqs]
    c = Case(hq=hq, hk=hk, d=d, kv=kv, q=(1,) * seqs, page=16, pad_rows=pad).upload()
    out, lse = with_canary(c, max_q=1, max_kv=3000)
    c.pool.sync()
    c.compare(out, lse, c.want())
    c.close()


@pytest.mark.parametrize("d,hq,hk", [(64, 16, 8), (576, 16, 1), (576, 64, 1)])
def test_sequences_that_are_named_twice(d, hq, hk):
    """A q_start that goes back between sequences is reported; the list of work is then longer than the launch,
    and what is left of it stays inside the workspace."""
    n = 20011
    c = Case(hq=hq, hk=hk, d=d, kv=(n,), q=(1,), page=64).upload()
    seqs = 33
    c.on["q_start"] = (torch.arange(seqs + 1) % 2).cuda()
    c.on["kv_len"] = torch.full((seqs,), n).cuda()
    c.on["table"] = c.table.expand(seqs, -1).contiguous().cuda()
    out, lse = with_canary(c, max_q=1, max_kv=n)
    with pytest.raises(B.HcError, match="lengths out of bounds; first flagged list position 1"):
        c.pool.sync()
    assert out.isfinite().all()
    c.close()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq", [17, 20, 32])
def test_latent_decoding_of_17_to_32_rows(hq, dtype):
    """Lengths around key tiles and splits, several tiles long."""
    check(dtype=dtype, hq=hq, hk=1, d=576, kv=(1, 2, 63, 64, 65, 127, 128, 129, 0, 300, 1500), q=(1,) * 11, page=24)


@pytest.mark.parametrize("kw", [dict(), dict(window=100, sinks=3), dict(window=1), dict(window=64, sinks=70),
                                dict(causal=False), dict(scale=-0.1), dict(scale=0.0)])
@pytest.mark.parametrize("hq,q", [(4, (8, 5, 1, 7)), (20, (1, 1, 1, 1)), (16, (2, 2, 1, 2)), (32, (1, 1, 1, 1))])
def test_latent_rows_of_several_tokens(hq, q, kw):
    """Windows and sinks across key tiles, rows of several tokens in a tile, long sequences that are split."""
    check(kw, hq=hq, hk=1, d=576, kv=(700, 65, 130, 2500), q=q, page=16, entry=1)


@pytest.mark.parametrize("hq,q", [(20, 1), (4, 8)])
def test_latent_maxima_that_grow(hq, q):
    """Scores that rise from key to key by far more than a tile's weights may grow before they are scaled, and fall."""
    c = Case(hq=hq, hk=1, d=576, kv=(500, 500, 333), q=(q, q, q), page=16, entry=1)
    for s, sign in ((0, 1.0), (1, -1.0), (2, 1.0)):
        where = F.slots_of(c.table[s], c.kv[s], 1)
        c.host[0][1, where, 512:] = (sign * torch.linspace(-1, 1, c.kv[s])[:, None] * torch.ones(64)).to(c.dt)
    c.q[..., 512:] = 12.0
    c.upload().check()
    c.close()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("hq,q", [(20, (1, 1)), (4, (8, 8)), (32, (1, 1))])
def test_latent_rows_that_do_not_see_what_is_not_finite(hq, q, bad):
    c = Case(hq=hq, hk=1, d=576, kv=(200, 1500), q=q, page=16)
    used = torch.zeros(c.host[0].shape[1], dtype=torch.bool)
    for s, n in enumerate(c.kv):
        used[F.slots_of(c.table[s], n, c.entry)] = True
    c.host[0][:, ~used] = bad
    for s in range(2):  # behind the window of every row, in the same tiles as what is seen
        where = F.slots_of(c.table[s], c.kv[s], c.entry)
        c.host[0][c.layer, where[40:c.kv[s] - 90]] = bad
    if q[1] > 1:  # the newest token: only its own rows see it
        c.host[0][c.layer, F.slots_of(c.table[1], 1500, c.entry)[-1]] = bad
    c.upload()
    kw = dict(window=80, sinks=35)
    out, lse = c.run(**kw)
    torch.cuda.synchronize()
    c.pool.sync()
    w, wl, tol, tol_l = c.want(**kw)
    n = int(c.q_start[-1]) - (1 if q[1] > 1 else 0)
    F.close(out[:n], w[:n], tol[:n], "out")
    F.close(lse[:n], wl[:n], tol_l[:n], "lse")
    assert out[:n].isfinite().all()
    c.close()
