"""Operators around a device KV pool that is held in 4 bits, as calls that can be measured.

Four kinds of call, in the order a serving step makes them:

  extend  pages for the new tokens of a batch, from the lengths of its sequences: table entries,
          the slot and position of every new token, row starts (``Pool.extend_pages``);
  axes    rotary positions with several axes (time, height, width) and the store of the tokens'
          keys and values in 16 bits (``Rope(sections=...)``, ``Pool.store_tokens``);
  store4  rotated keys and values stored in 4 bits, and the stored rows read back as elements
          (``Pool.store_tokens(cache="mxfp4")``, ``Pool.fetch_tokens``);
  attend4 attention of a chunk of new tokens (one token while decoding) over the cached tokens of
          a 4-bit cache (``Pool.attend(cache="mxfp4")``).

A 4-bit row holds codes of all its elements (two a byte, the lower half first), then a scale byte
for every 32 of them, and is rounded up to 16 bytes.  A value is sign * {0, 0.5, 1, 1.5, 2, 3, 4, 6}
* 2^(scale - 127).  The scale is the least that keeps the block's largest value within 7 of it, so
that no value is off by more than half a step.

``run`` computes a call in its plain form, in elementary torch operations, unless ``own`` is
set: then it makes the library's call.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 32


# ---------------------------------------------------------------- cases
def _store(**kw):
    base = dict(op="store4", dtype="bf16", q_heads=32, kv_heads=8, head=128, value=128, rot=128, rot_offset=0,
                interleaved=False, base=500000.0, llama3=0.0, original=8192, tokens=32, far=32768, slots=16384, page=64,
                sections="", cyclic=False, own_series=False)
    base.update(kw)
    return base


def _attend(**kw):
    base = dict(op="attend4", dtype="bf16", q_heads=32, kv_heads=8, head=128, value=128, page=64, entry=64, batch=1,
                q_len=1, kv_len=1024, ragged=False, causal=True, window=0, sinks=0, lse=False)
    base.update(kw)
    return base


def _latent(**kw):
    return dict(_attend(kv_heads=1, q_heads=16, head=576, value=512), **kw)


def _extend(**kw):
    base = dict(op="extend", page=64, sequences=64, kv_len=8192, prompts=0, prompt=1, spare=0)
    base.update(kw)
    return base


def listed():
    return [
        # one decoding step of 32 conversations about images: a token stands at one place on every axis
        dict(_store(op="axes", tokens=32, sections="16,24,24", base=1000000.0), name="axes_store_decode_32"),
        # the frames of a clip in one prefill step: time, height and width
        dict(_store(op="axes", tokens=8192, slots=32768, sections="16,24,24", base=1000000.0), name="axes_store_video_8192"),
        # one decoding step of 32 sequences into a 4-bit cache, 32 query and 8 KV heads of 128
        dict(_store(tokens=32, llama3=8.0, far=131072), name="store4_decode_32"),
        # the prompt tokens of one prefill step
        dict(_store(tokens=8192, slots=32768, llama3=8.0), name="store4_prompt_8192"),
        # one token of one conversation: latency
        dict(_attend(kv_len=1500), name="attend4_decode_1x1500"),
        # a decoding batch of unequal lengths over pages
        dict(_attend(batch=64, kv_len=8192, ragged=True), name="attend4_decode_64x8192"),
        # long sequences seen through a window, slots scattered token by token, fp16 heads of 64
        dict(_attend(batch=32, kv_len=32768, q_heads=16, kv_heads=8, head=64, value=64, dtype="fp16", page=16, entry=1,
                     window=4096, sinks=4, ragged=True, lse=True), name="attend4_window_32x32768"),
        # a chunk of a long prompt behind its cached prefix
        dict(_attend(q_len=2048, kv_len=16384), name="attend4_chunk_2048_16384"),
        # decoding over a latent cache, 16 heads on this GPU
        dict(_latent(batch=32, kv_len=6000, ragged=True), name="attend4_latent_32x6000"),
        # a chunk over a latent cache
        dict(_latent(q_len=512, kv_len=4500, q_heads=32), name="attend4_latent_chunk_512"),
        # the next token of 64 sequences
        dict(_extend(), name="extend_decode_64"),
        # prompts of unequal lengths beside decoding sequences, a batch padded to its graph's size
        dict(_extend(sequences=512, kv_len=32768, prompts=64, prompt=2048, spare=1000), name="extend_mixed_512"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["axes", "store4", "store4", "attend4", "attend4", "attend4", "extend"])
    if op in ("axes", "store4"):
        latent = op == "store4" and rng.random() < 0.3
        head = 576 if latent else rng.choice([64, 96, 128, 256])
        rot = 64 if latent else rng.choice([r for r in (32, 64, 96, 128, 256) if r <= head])
        kv_heads = 1 if latent else rng.choice([1, 2, 4, 8])
        axes = rng.choice([2, 3]) if op == "axes" or rng.random() < 0.4 else 0
        cuts = sorted(rng.sample(range(1, rot // 2), axes - 1)) if axes else []
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])] if axes else []
        own_series = bool(axes) and rng.random() < 0.3
        return _store(op=op, tokens=_log(rng, 1, 8192), q_heads=kv_heads * rng.choice([1, 4, 7, 8]), kv_heads=kv_heads,
                      head=head, value=0 if latent else head, rot=rot, rot_offset=512 if latent else 0,
                      interleaved=latent or rng.random() < 0.3, base=rng.choice([10000.0, 500000.0]),
                      llama3=0.0 if own_series else rng.choice([0.0, 8.0, 32.0]), dtype=rng.choice(["bf16", "fp16"]),
                      far=_log(rng, 100, 1000000), page=rng.choice([16, 64]), sections=",".join(map(str, sections)),
                      cyclic=bool(axes) and not own_series and rng.random() < 0.3, own_series=own_series)
    if op == "attend4":
        latent = rng.random() < 0.3
        decode = rng.random() < 0.5
        kv_heads = 1 if latent else rng.choice([1, 2, 4, 8])
        group = rng.choice([8, 16, 20, 128]) if latent else rng.choice([1, 2, 3, 4, 7, 8, 16])
        head = 576 if latent else rng.choice([64, 128])
        page = rng.choice([16, 24, 64])
        batch = _log(rng, 1, 64)
        kv_len = _log(rng, 1, 32768)
        q_len = 1 if decode else min(kv_len, _log(rng, 2, 4096))
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        case = _attend(dtype=rng.choice(["bf16", "fp16"]), q_heads=kv_heads * group, kv_heads=kv_heads, head=head,
                       value=512 if latent else head, page=page, entry=rng.choice([1, page]), batch=batch,
                       q_len=q_len, kv_len=kv_len, ragged=rng.random() < 0.7, causal=decode or rng.random() < 0.8,
                       window=window, sinks=rng.choice([0, 4, 33]) if window else 0, lse=rng.random() < 0.3)
        case["causal"] = case["causal"] or window > 0
        # no more work, and no larger score matrix, than the listed cases have
        while (work(dict(case, ragged=False, window=0))["flops"] > 4e11
               or case["batch"] * case["kv_len"] * (case["q_heads"] * case["q_len"] + 2 * kv_heads * head) > 1.2e9):
            if case["batch"] > 1:
                case["batch"] = (case["batch"] + 1) // 2
            elif case["q_len"] > 1:
                case["q_len"] = (case["q_len"] + 1) // 2
            else:
                case["kv_len"] = (case["kv_len"] + 1) // 2
            case["q_len"] = min(case["q_len"], case["kv_len"])
        return case
    sequences = _log(rng, 1, 512)
    return _extend(page=rng.choice([16, 24, 64]), sequences=sequences, kv_len=_log(rng, 1, 32768),
                   prompts=rng.randint(0, min(sequences, 64)), prompt=_log(rng, 1, 2048), spare=_log(rng, 1, 1000))


# ---------------------------------------------------------------- sizes that follow from a case alone
def _spread(n, longest, ragged):
    """n lengths: all the longest, or spread evenly up to it."""
    return [max(1, longest * (i + 1) // n) if ragged else longest for i in range(n)]


def _seen(case, q, kv):
    """Visible (query, key) pairs of one sequence and keys that any query sees."""
    first, w = kv - q, case["window"]
    if not case["causal"]:
        return q * kv, kv
    pairs = sum(min(p + 1, w + min(case["sinks"], max(0, p + 1 - w)) if w else p + 1) for p in range(first, kv))
    low = max(0, first + 1 - w) if w else 0
    return pairs, kv - low + min(low, case["sinks"])


def _grown(case):
    """Cached and new tokens of each sequence: prompts first, then one token each."""
    lens = _spread(case["sequences"], case["kv_len"], True)
    added = _spread(max(1, case["prompts"]), case["prompt"], True)[: case["prompts"]]
    return lens, added + [1] * (case["sequences"] - case["prompts"])


def work(case):
    if case["op"] in ("axes", "store4"):
        n, q, kv = case["tokens"], case["q_heads"] * case["head"], case["kv_heads"] * (case["head"] + case["value"])
        lists = 8 * n * (1 + max(1, len(case["sections"].split(","))))
        # in 4 bits: read, stored, read back, written as elements
        moved = 4 * q + (4 * kv if case["op"] == "axes" else 4 * kv + 2 * kv * 17 / 32)
        return {"bytes": n * moved + lists, "flops": 3 * n * (case["q_heads"] + case["kv_heads"]) * case["rot"]}
    if case["op"] == "attend4":
        kv = _spread(case["batch"], case["kv_len"], case["ragged"])
        q = [min(a, b) for a, b in zip(_spread(case["batch"], case["q_len"], case["ragged"]), kv)]
        seen = [_seen(case, a, b) for a, b in zip(q, kv)]
        row = case["kv_heads"] * (case["head"] + (0 if case["head"] == 576 else case["value"])) * 17 / 32
        io = sum(q) * case["q_heads"] * (case["head"] + case["value"])
        return {"bytes": row * sum(k for _, k in seen) + 2 * io + 8 * sum(b // case["entry"] for b in kv),
                "flops": 2 * case["q_heads"] * (case["head"] + case["value"]) * sum(p for p, _ in seen)}
    lens, added = _grown(case)
    pages = sum(-(-(a + b) // case["page"]) - -(-a // case["page"]) for a, b in zip(lens, added))
    return {"bytes": 32 * len(lens) + 16 * (sum(added) + case["spare"]) + 16 * pages, "flops": 0}


def _row_bytes(heads, dim):
    n = heads * dim
    return -(-(n // 2 + n // BLOCK) // 16) * 16


# ---------------------------------------------------------------- inputs
def _pool(state, subs, slots, page):
    """The pool handle a serving program creates once; subs: bytes of a row."""
    from host_device_page_amd import binding as B

    buffers = state["pool"]
    state["handle"] = B.Pool(layers=2, page_size=page, subs=[(B.HC_TOKEN_ROWS, e) for e in subs],
                             device_slots=slots, host_pages=0, device_layers=[[t[0], t[1]] for t in buffers],
                             host=None, stream=torch.cuda.current_stream())
    return B


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case.get("dtype", "bf16")]

    def normal(*shape, scale=1.0):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(0.0, scale, generator=g)

    def shuffled(n):
        return torch.randperm(n, generator=g, device="cuda")

    state = dict(case=case)
    if case["op"] in ("axes", "store4"):
        n, hq, hk, d, dv, slots = (case[k] for k in ("tokens", "q_heads", "kv_heads", "head", "value", "slots"))
        parts = [hk * d] + ([hk * dv] if dv else [])
        axes = len(case["sections"].split(",")) if case["sections"] else 0
        if axes:
            # a clip: the first axis counts frames, the others places inside one
            i = torch.arange(n, device="cuda")
            start = torch.randint(0, case["far"], (1,), generator=g, device="cuda")
            side = max(1, int(math.sqrt(n) / 2))
            place = [i // (side * side), i // side % side, i % side]
            positions = start + torch.stack(place[3 - axes:])
        else:
            positions = torch.randint(0, case["far"], (n,), generator=g, device="cuda")
        k, v = normal(n, hk, d), normal(n, hk, dv) if dv else None
        if case["op"] == "store4":  # channels of unlike size, as keys have them
            k = k * torch.exp(torch.empty((hk, d), device="cuda").normal_(0.0, 1.0, generator=g)).to(dt)
        state.update(q=normal(n, hq, d), k=k, v=v, q_out=torch.empty((n, hq, d), dtype=dt, device="cuda"),
                     positions=positions.contiguous(), slots=shuffled(slots)[:n].contiguous())
        if case["op"] == "store4":
            subs = [_row_bytes(hk, e // hk) for e in parts]
            state.update(pool=[torch.zeros((2, slots, e), dtype=torch.uint8, device="cuda") for e in subs],
                         back=[torch.empty((n, hk, e // hk), dtype=dt, device="cuda") for e in parts])
        else:
            subs = [2 * e for e in parts]
            state.update(pool=[normal(2, slots, e) for e in parts])
        if own:
            B = _pool(state, subs, slots, case["page"])
            state["rope"] = B.Rope(rot_dim=case["rot"], base=case["base"], interleaved=case["interleaved"],
                                   rot_offset=case["rot_offset"], **_scaling(case), **_axes_of(case))
        return state
    if case["op"] == "attend4":
        b, hq, hk, d, dv, page, entry = (case[k] for k in ("batch", "q_heads", "kv_heads", "head", "value", "page", "entry"))
        kv = _spread(b, case["kv_len"], case["ragged"])
        q = [min(x, y) for x, y in zip(_spread(b, case["q_len"], case["ragged"]), kv)]
        order = shuffled(b).tolist()
        kv, q = [kv[i] for i in order], [q[i] for i in order]
        used = [-(-n // page) for n in kv]
        pages = sum(used) + 1 + sum(used) // 8
        width = -(-case["kv_len"] // entry)
        kv_len = torch.tensor(kv, device="cuda")
        each = torch.arange(width, device="cuda")
        live = each[None, :] < ((kv_len + entry - 1) // entry)[:, None]
        # every sequence's entries, in random places of the pool; what lies behind a sequence is not an entry
        place = shuffled(pages * page // entry)
        table = torch.full((b, width), -1, dtype=torch.int64, device="cuda")
        table[live] = place[: int(live.sum())]
        heads = [(hk, d)] + ([] if d == 576 else [(hk, dv)])
        state.update(pool=[_cache(g, 2, pages * page, *x) for x in heads], table=table, kv_len=kv_len,
                     q=normal(sum(q), hq, d, scale=2.0),
                     q_start=torch.tensor([0] + q, device="cuda").cumsum(0),
                     out=torch.empty((sum(q), hq, dv), dtype=dt, device="cuda"))
        if own:
            _pool(state, [_row_bytes(*x) for x in heads], pages * page, page)
        return state
    page = case["page"]
    lens, added = _grown(case)
    order = shuffled(len(lens)).tolist()
    lens, added = [lens[i] for i in order], [added[i] for i in order]
    held = [-(-n // page) for n in lens]
    wanted = sum(-(-(a + b) // page) - h for a, b, h in zip(lens, added, held))
    pages = sum(held) + wanted + 9
    width = -(-(case["kv_len"] + case["prompt"]) // page)
    held = torch.tensor(held, device="cuda")
    live = torch.arange(width, device="cuda")[None, :] < held[:, None]
    place = shuffled(pages)
    table = torch.full((len(lens), width), -1, dtype=torch.int64, device="cuda")
    table[live] = place[: int(live.sum())]
    state.update(table=table, lens=torch.tensor(lens, device="cuda"), added=torch.tensor(added, device="cuda"),
                 free=place[int(live.sum()):].contiguous(), room=sum(added) + case["spare"],
                 pool=[torch.zeros((2, pages * page, 16), dtype=torch.uint8, device="cuda")])
    if own:
        _pool(state, [16], pages * page, page)
    return state


def _cache(g, layers, slots, heads, dim):
    """4-bit rows of normal keys or values whose channels differ in size."""
    rows = torch.zeros((layers, slots, _row_bytes(heads, dim)), dtype=torch.uint8, device="cuda")
    size = torch.exp(torch.empty((heads * dim,), device="cuda").normal_(0.0, 0.5, generator=g))
    for layer in range(layers):
        for at in range(0, slots, 1 << 16):
            part = rows[layer, at:at + (1 << 16)]
            x = torch.empty((part.shape[0], heads * dim), device="cuda").normal_(0.0, 1.0, generator=g) * size
            part.copy_(_pack(x))
    return rows


def _scaling(case):
    return dict(scaling="llama3", factor=case["llama3"], original_context=case["original"]) if case["llama3"] else {}


def _axes_of(case):
    """How the pairs of a rotation are shared out over its axes, as arguments of a Rope."""
    if not case["sections"]:
        return {}
    sections = [int(x) for x in case["sections"].split(",")]
    if case["cyclic"]:
        return dict(pair_axes=[i % len(sections) for i in range(case["rot"] // 2)])
    return dict(sections=sections, own_series=case["own_series"])


# ---------------------------------------------------------------- plain forms
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _power(e, dtype):
    """2^e, of whole numbers."""
    if dtype == torch.float64:
        return ((e.long() + 1023) << 52).view(torch.float64)
    return torch.exp2(e.to(dtype))


def _pack(x):
    """Rows of 4-bit codes and scales for rows of elements (n, elements)."""
    n, elements = x.shape
    block = x.double().view(n, elements // BLOCK, BLOCK)  # 64 bits: values next to a border
    fraction, exponent = torch.frexp(block.abs().amax(-1))
    scale = torch.where(fraction <= 0.875, exponent - 3, exponent - 2).clamp(-127, 127)
    size = (block * _power(-scale, torch.float64)[..., None]).abs()
    code = torch.zeros(size.shape, dtype=torch.uint8, device=x.device)
    # halfway goes to the even code
    code += size > 0.25
    code += size >= 0.75
    code += size > 1.25
    code += size >= 1.75
    code += size > 2.5
    code += size >= 3.5
    code += size > 5.0
    code = (code + 8 * (block < 0).to(torch.uint8)).view(n, elements)
    rows = torch.zeros((n, _row_bytes(1, elements)), dtype=torch.uint8, device=x.device)
    rows[:, : elements // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    rows[:, elements // 2: elements // 2 + elements // BLOCK] = (scale + 127).to(torch.uint8)
    return rows


def _unpack(rows, elements):
    """The elements of 4-bit rows (..., bytes), in 32 bits."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=rows.device)
    codes = rows[..., : elements // 2]
    value = table[torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).int()]
    scale = _power(rows[..., elements // 2: elements // 2 + elements // BLOCK].float() - 127.0, torch.float32)
    return (value.unflatten(-1, (-1, BLOCK)) * scale[..., None]).flatten(-2)


def _frequencies(case):
    """Radians per position of each rotated pair, and the axis whose position it takes."""
    n = case["rot"] // 2
    i = torch.arange(n, dtype=torch.float64, device="cuda")
    f = torch.exp(-math.log(case["base"]) * i / n)
    axis = torch.zeros(n, dtype=torch.int64, device="cuda")
    if case["sections"]:
        sections = torch.tensor([int(x) for x in case["sections"].split(",")], device="cuda")
        axis = torch.repeat_interleave(torch.arange(len(sections), device="cuda"), sections)
        if case["own_series"]:  # every axis counts its own pairs
            first = (sections.cumsum(0) - sections)[axis]
            f = torch.exp(-math.log(case["base"]) * (i - first) / sections[axis])
        if case["cyclic"]:
            axis = torch.arange(n, device="cuda") % len(sections)
    if case["llama3"]:
        turns = case["original"] * f / (2 * math.pi)  # over the original context; kept above 4, divided below 1
        keep = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
        f = f * (keep + (1 - keep) / case["llama3"])
    return f, axis


def _rotated(case, x, positions, dtype):
    """Rotated heads, computed in `dtype`."""
    f, axis = _frequencies(case)
    angle = torch.atleast_2d(positions).double().t()[:, axis] * f  # 64 bits: far positions
    cos, sin = angle.cos().to(dtype)[:, None], angle.sin().to(dtype)[:, None]
    a, r = case["rot_offset"], case["rot"]
    part = x[..., a:a + r].to(dtype)
    if case["interleaved"]:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1).flatten(-2)
    else:
        x1, x2 = part[..., : r // 2], part[..., r // 2:]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)
    return torch.cat([x[..., :a].to(dtype), turned, x[..., a + r:].to(dtype)], dim=-1)


def _plain_store(s):
    case, slots, positions = s["case"], s["slots"], s["positions"]
    s["q_out"].copy_(_rotated(case, s["q"], positions, torch.float32))
    if case["op"] == "axes":
        s["pool"][0][1].index_copy_(0, slots, _rotated(case, s["k"], positions, torch.float32).to(s["k"].dtype).flatten(1))
        s["pool"][1][1].index_copy_(0, slots, s["v"].flatten(1))
        return
    s["pool"][0][1].index_copy_(0, slots, _pack(_rotated(case, s["k"], positions, torch.float64).flatten(1)))
    if s["v"] is not None:
        s["pool"][1][1].index_copy_(0, slots, _pack(s["v"].flatten(1)))
    s["back"][0].copy_(_unpack(s["pool"][0][1][slots], s["k"][0].numel()).view_as(s["k"]))
    if s["v"] is not None:
        s["back"][1].copy_(_unpack(s["pool"][1][1][slots], s["v"][0].numel()).view_as(s["v"]))


def _visible(case, position, key):
    if not case["causal"]:
        return (key >= 0) & (position >= position)
    seen = key <= position
    if case["window"]:
        seen = seen & ((position - key < case["window"]) | (key < case["sinks"]))
    return seen


def _plain_attend(s):
    case = s["case"]
    b, hq, hk, d, dv, e = (case[k] for k in ("batch", "q_heads", "kv_heads", "head", "value", "entry"))
    m, n, t = case["q_len"], case["kv_len"], s["q"].shape[0]
    key = torch.arange(n, device="cuda")
    slot = (s["table"].clamp(min=0)[:, key // e] * e + key % e)
    there = key[None] < s["kv_len"][:, None]
    slot = torch.where(there, slot, 0)
    # the packed queries, laid out one block of m rows a sequence
    row = torch.arange(t, device="cuda")
    seq = torch.searchsorted(s["q_start"], row, right=True) - 1
    at = row - s["q_start"][seq]
    q = torch.zeros((b, m, hq, d), device="cuda")
    q[seq, at] = s["q"].float()
    count = (s["q_start"][1:] - s["q_start"][:-1])
    position = s["kv_len"][:, None] - count[:, None] + torch.arange(m, device="cuda")[None]
    k = _unpack(s["pool"][0][1][slot], hk * d).view(b, n, hk, d)
    v = k[..., :dv] if d == 576 else _unpack(s["pool"][1][1][slot], hk * dv).view(b, n, hk, dv)
    k = k.permute(0, 2, 3, 1).contiguous()  # b hk d n
    q = q.view(b, m, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)  # b hk (group m) d
    score = torch.matmul(q, k).view(b, hk, hq // hk, m, n).mul_(d ** -0.5)
    seen = _visible(case, position[:, :, None], key) & there[:, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    v = v.permute(0, 2, 1, 3).contiguous()
    out = torch.matmul(score.view(b, hk, -1, n), v).view(b, hk, hq // hk, m, dv)
    out = (out / torch.where(total == 0, 1.0, total)).permute(0, 3, 1, 2, 4).reshape(b, m, hq, dv)
    s["out"].copy_(out[seq, at].to(s["out"].dtype))
    if not case["lse"]:
        return None
    return (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(b, m, hq)[seq, at]


def _plain_extend(s):
    p, lens, added, table = s["case"]["page"], s["lens"], s["added"], s["table"]
    kv_len = lens + added
    held = (lens + p - 1) // p
    fresh = (kv_len + p - 1) // p - held
    first = fresh.cumsum(0) - fresh
    q_start = torch.cat([added.new_zeros(1), added.cumsum(0)])
    column = torch.arange(table.shape[1], device="cuda")[None]
    new = (column >= held[:, None]) & (column < (held + fresh)[:, None])
    place = (first - held)[:, None] + column
    table.copy_(torch.where(new, s["free"][torch.where(new, place, 0)], table))
    row = torch.arange(s["room"], device="cuda")
    seq = (torch.searchsorted(q_start, row, right=True) - 1).clamp(max=len(lens) - 1)
    live = row < q_start[-1]
    position = torch.where(live, lens[seq] + row - q_start[seq], 0)
    slots = torch.where(live, table[seq, position // p] * p + position % p, -1)
    return kv_len, q_start, slots, position, fresh.sum()[None]


# ---------------------------------------------------------------- one call
def run(state):
    case = state["case"]
    if case["op"] in ("axes", "store4"):
        if own:
            kw = dict(cache="mxfp4") if case["op"] == "store4" else {}
            state["handle"].store_tokens(1, state["slots"], state["k"], state["v"], q=state["q"], q_out=state["q_out"],
                                         rope=state["rope"], positions=state["positions"], **kw)
            if case["op"] == "store4":
                back = state["back"]
                state["handle"].fetch_tokens(1, state["slots"], back[0], back[1] if len(back) > 1 else None)
        else:
            _plain_store(state)
        if case["op"] == "axes":
            return {"q": state["q_out"], "pool": state["pool"]}
        return {"q": state["q_out"], "values": state["back"]}
    if case["op"] == "attend4":
        if own:
            lse = state["handle"].attend(1, state["q"], state["table"], state["kv_len"], q_start=state["q_start"],
                                         kv_heads=case["kv_heads"], max_q=case["q_len"], max_kv=case["kv_len"],
                                         entry_tokens=case["entry"], causal=case["causal"], window=case["window"],
                                         sinks=case["sinks"], out=state["out"], return_lse=case["lse"],
                                         cache="mxfp4")[1]
        else:
            lse = _plain_attend(state)
        return {"out": state["out"], "lse": lse} if case["lse"] else {"out": state["out"]}
    if own:
        got = state["handle"].extend_pages(state["table"], state["lens"], state["added"], state["free"],
                                           tokens=state["room"])
    else:
        got = _plain_extend(state)
    return dict(zip(("kv_len", "q_start", "slots", "positions", "used"), got), table=state["table"])


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_turn(case, x, positions):
    pairs = case["rot"] // 2
    sections = [int(v) for v in case["sections"].split(",")] if case["sections"] else [pairs]
    theta, axis = [], []
    for i in range(pairs):
        a, j = 0, i
        while j >= sections[a]:
            j -= sections[a]
            a += 1
        share = j / sections[a] if case["own_series"] else i / pairs
        f = case["base"] ** -share
        if case["llama3"]:
            wave = 2 * math.pi / f
            if wave > case["original"]:
                f /= case["llama3"]
            elif wave > case["original"] / 4:
                smooth = (case["original"] / wave - 1) / 3
                f = (1 - smooth) * f / case["llama3"] + smooth * f
        theta.append(f)
        axis.append(i % len(sections) if case["cyclic"] else a)
    where = positions.view(len(sections), -1).double()[axis].t()
    angle = where * torch.tensor(theta, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.double().clone()
    a, h = case["rot_offset"], pairs
    first = slice(a, a + 2 * h, 2) if case["interleaved"] else slice(a, a + h)
    second = slice(a + 1, a + 2 * h, 2) if case["interleaved"] else slice(a + h, a + 2 * h)
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _exact_values(x):
    """What x is stored as: its blocks on the grid of their scales."""
    block = x.flatten(1).unflatten(1, (-1, BLOCK))
    top = block.abs().amax(-1, keepdim=True)
    step = torch.exp2(torch.ceil(torch.log2(top / 7)))
    step = torch.where(top > 7 * step, 2 * step, step)
    step = torch.where(top <= 3.5 * step, step / 2, step)
    size = (block / step).abs()
    grid = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
    size = (torch.round(size / grid) * grid).clamp(max=6.0)  # round: halfway to even
    return (size * step * torch.sign(block)).view_as(x)


def _exact_rows(rows, elements):
    """The elements of 4-bit rows, from the bits of each code."""
    codes = torch.repeat_interleave(rows[:, : elements // 2].long(), 2, dim=1)
    codes = torch.where(torch.arange(elements, device="cuda") % 2 == 1, codes // 16, codes % 16)
    exponent, mantissa = codes // 2 % 4, codes % 2
    size = torch.where(exponent == 0, mantissa * 0.5, (2 + mantissa) * 2.0 ** (exponent - 2).double())
    scale = rows[:, elements // 2: elements // 2 + elements // BLOCK].double() - 127
    return torch.where(codes >= 8, -size, size) * torch.repeat_interleave(torch.exp2(scale), BLOCK, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("axes", "store4"):
        q, k = (_exact_turn(case, s[x], s["positions"]) for x in ("q", "k"))
        if case["op"] == "store4":
            v = [] if s["v"] is None else [_exact_values(s["v"].double())]
            return {"q": q, "values": [_exact_values(k)] + v}
        pool = [t.double() for t in s["pool"]]
        pool[0][1, s["slots"]] = k.flatten(1)
        pool[1][1, s["slots"]] = s["v"].double().flatten(1)
        return {"q": q, "pool": pool}
    if case["op"] == "attend4":
        hk, d, dv, e = (case[k] for k in ("kv_heads", "head", "value", "entry"))
        group = case["q_heads"] // hk
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["out"].shape[:2], dtype=torch.float64, device="cuda")
        start, lens = s["q_start"].tolist(), s["kv_len"].tolist()
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            rows = s["table"][b][j // e] * e + j % e
            keys = _exact_rows(s["pool"][0][1][rows], hk * d)
            values = keys if d == 576 else _exact_rows(s["pool"][1][1][rows], hk * dv)
            for h in range(hk):
                kt = keys[:, h * d:(h + 1) * d].t().contiguous()
                v = values[:, :dv] if d == 576 else values[:, h * dv:(h + 1) * dv]
                for r in range(start[b], start[b + 1], 1024):
                    stop = min(r + 1024, start[b + 1])
                    p = n - (start[b + 1] - torch.arange(r, stop, device="cuda"))[:, None, None]
                    x = torch.matmul(s["q"][r:stop, h * group:(h + 1) * group].double(), kt) / math.sqrt(d)
                    if case["causal"]:
                        hidden = j > p
                        if case["window"]:
                            hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
                        x = x.masked_fill(hidden, -math.inf)
                    out[r:stop, h * group:(h + 1) * group] = torch.matmul(torch.softmax(x, -1), v.contiguous())
                    lse[r:stop, h * group:(h + 1) * group] = torch.logsumexp(x, -1)
        return {"out": out, "lse": lse} if case["lse"] else {"out": out}
    # whole numbers, sequence by sequence
    p, free, taken, q_start, slots, positions, kv_len, rows = case["page"], s["free"].tolist(), 0, [0], [], [], [], []
    for row, n, m in zip(s["table"].tolist(), s["lens"].tolist(), s["added"].tolist()):
        for j in range(n, n + m):
            if j % p == 0:
                row[j // p] = free[taken]
                taken += 1
            slots.append(row[j // p] * p + j % p)
            positions.append(j)
        rows.append(row)
        kv_len.append(n + m)
        q_start.append(q_start[-1] + m)
    pad = s["room"] - len(slots)
    got = dict(kv_len=kv_len, q_start=q_start, slots=slots + [-1] * pad, positions=positions + [0] * pad, used=[taken], table=rows)
    return {k: torch.tensor(v) for k, v in got.items()}
