"""The operators that a forward pass runs on a device KV pool, as calls that can be measured.

Three kinds of call, in the order a serving step makes them:

  store   rotary positions on queries and keys, the rotated keys and the values written into
          their token slots of one layer (``Pool.store_tokens``);
  attend  attention of a chunk of new tokens (one token while decoding) over the cached tokens
          of its sequence, optionally through a sliding window with a few first tokens that
          stay visible (``Pool.attend``);
  fork / compact
          page tables of forked sequences with a copy of each partly filled last page
          (``Pool.fork_pages``), and the live pages moved to the front of the pool
          (``Pool.compact_pages``), over all layers.

``run`` computes a call in its plain form, in elementary torch operations, unless ``own`` is
set: then it makes the library's call.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def _store(**kw):
    base = dict(op="store", dtype="bf16", q_heads=32, kv_heads=8, head=128, value=128, rot=128, rot_offset=0,
                interleaved=False, base=500000.0, scaling="none", factor=1.0, original=8192, tokens=32,
                far=32768, slots=16384, page=64)
    base.update(kw)
    return base


def _attend(**kw):
    base = dict(op="attend", dtype="bf16", q_heads=32, kv_heads=8, head=128, value=128, page=64, entry=64, batch=1,
                q_len=1, kv_len=1024, ragged=False, causal=True, window=0, sinks=0, lse=False)
    base.update(kw)
    return base


def _latent(**kw):
    return dict(_attend(kv_heads=1, q_heads=16, head=576, value=512), **kw)


def listed():
    return [
        # one decoding step of 32 sequences, 32 query and 8 KV heads of 128
        dict(_store(tokens=32, scaling="llama3", factor=8.0, far=131072), name="store_decode_32"),
        # the prompt tokens of one prefill step
        dict(_store(tokens=8192, slots=32768, scaling="llama3", factor=8.0), name="store_prompt_8192"),
        # a chunk of a latent cache: 64 rotated dims behind 512, interleaved pairs, a stretched context
        dict(_store(tokens=2048, q_heads=16, kv_heads=1, head=576, value=0, rot=64, rot_offset=512, interleaved=True,
                    base=10000.0, scaling="yarn", factor=40.0, original=4096, far=160000), name="store_latent_2048"),
        # one token of one conversation: latency
        dict(_attend(kv_len=1500), name="attend_decode_1x1500"),
        # a decoding batch of unequal lengths over pages
        dict(_attend(batch=64, kv_len=8192, ragged=True), name="attend_decode_64x8192"),
        # long sequences seen through a window, slots scattered token by token, fp16 heads of 64
        dict(_attend(batch=32, kv_len=32768, q_heads=16, kv_heads=8, head=64, value=64, dtype="fp16", page=16, entry=1,
                     window=4096, sinks=4, ragged=True, lse=True), name="attend_window_32x32768"),
        # a chunk of a long prompt behind its cached prefix
        dict(_attend(q_len=2048, kv_len=16384), name="attend_chunk_2048_16384"),
        # prompts of unequal lengths computed whole, fp16 heads of 64
        dict(_attend(batch=4, q_len=4096, kv_len=4096, q_heads=16, kv_heads=4, head=64, value=64, dtype="fp16",
                     ragged=True, page=32, entry=32), name="attend_prompts_4x4096"),
        # decoding over the latent cache, 16 heads on this GPU
        dict(_latent(batch=32, kv_len=6000, ragged=True), name="attend_latent_32x6000"),
        # a chunk over the latent cache
        dict(_latent(q_len=512, kv_len=4500, q_heads=32), name="attend_latent_chunk_512"),
        # 64 samples branched off 8 prompts of unequal lengths, 32 layers
        dict(op="fork", dtype="bf16", layers=32, page=64, row=2048, parents=8, children=64, kv_len=2000, pages=512,
             name="fork_64_of_8"),
        # a fragmented pool packed: every third page live
        dict(op="compact", dtype="bf16", layers=8, page=64, row=2048, sequences=24, kv_len=1100, pages=1024,
             name="compact_1024_pages"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["store", "attend", "attend", "attend", "fork", "compact"])
    if op == "store":
        latent = rng.random() < 0.3
        scaling = rng.choice(["none", "linear", "llama3", "yarn"])
        head = 576 if latent else rng.choice([64, 96, 128, 256])
        rot = 64 if latent else rng.choice([r for r in (32, 64, 96, 128, 256) if r <= head])
        kv_heads = 1 if latent else rng.choice([1, 2, 4, 8])
        return _store(tokens=_log(rng, 1, 8192), q_heads=kv_heads * rng.choice([1, 4, 7, 8]), kv_heads=kv_heads,
                      head=head, value=0 if latent else head, rot=rot, rot_offset=512 if latent else 0,
                      interleaved=latent or rng.random() < 0.3, base=rng.choice([10000.0, 500000.0]), scaling=scaling,
                      factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 40.0]),
                      dtype=rng.choice(["bf16", "fp16"]), far=_log(rng, 100, 1000000), page=rng.choice([16, 64]))
    if op == "attend":
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
    page = rng.choice([16, 64])
    if op == "fork":
        parents = rng.randint(1, 8)
        kv_len = _log(rng, 1, 2000)
        children = _log(rng, 1, 64)
        return dict(op="fork", dtype="bf16", layers=rng.choice([4, 16, 32]), page=page, row=rng.choice([1024, 2048, 1152]),
                    parents=parents, children=children, kv_len=kv_len,
                    pages=parents * (kv_len // page + 1) + children + rng.randint(1, 40))
    sequences = rng.randint(1, 24)
    kv_len = _log(rng, 1, 1100)
    used = sequences * (kv_len // page + 1)
    return dict(op="compact", dtype="bf16", layers=rng.choice([2, 5, 8]), page=page, row=rng.choice([1024, 2048, 1152]),
                sequences=sequences, kv_len=kv_len, pages=used + _log(rng, 1, max(2, min(2 * used, 600))))


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


def work(case):
    if case["op"] == "store":
        n, h = case["tokens"], case["head"]
        moved = n * (2 * case["q_heads"] * h + 2 * case["kv_heads"] * h + 2 * case["kv_heads"] * case["value"])
        return {"bytes": 2 * moved + 16 * n, "flops": 3 * n * (case["q_heads"] + case["kv_heads"]) * case["rot"]}
    if case["op"] == "attend":
        kv = _spread(case["batch"], case["kv_len"], case["ragged"])
        q = [min(a, b) for a, b in zip(_spread(case["batch"], case["q_len"], case["ragged"]), kv)]
        seen = [_seen(case, a, b) for a, b in zip(q, kv)]
        row = case["kv_heads"] * (case["head"] + (0 if case["head"] == 576 else case["value"]))
        io = sum(q) * case["q_heads"] * (case["head"] + case["value"])
        return {"bytes": 2 * (row * sum(k for _, k in seen) + io) + 8 * sum(b // case["entry"] for b in kv),
                "flops": 2 * case["q_heads"] * (case["head"] + case["value"]) * sum(p for p, _ in seen)}
    if case["op"] == "fork":
        lens = _spread(case["parents"], case["kv_len"], True)
        rows = sum(lens[i % len(lens)] % case["page"] for i in range(case["children"]))
        moved = rows * case["layers"] * 2 * case["row"]
        return {"bytes": 2 * moved + 16 * case["children"] * (case["kv_len"] // case["page"] + 1), "flops": 0}
    live = _live(case)
    moved = live * (case["pages"] - live) // case["pages"]  # live pages above the packed end, on average
    return {"bytes": 2 * moved * case["layers"] * case["page"] * 2 * case["row"] + 16 * live, "flops": 0}


def _live(case):
    return sum(-(-n // case["page"]) for n in _spread(case["sequences"], case["kv_len"], True))


# ---------------------------------------------------------------- inputs
def _pool(state, subs, layers, slots, page):
    """The pool handle a serving program creates once."""
    from host_device_page_amd import binding as B

    buffers = state["pool"]
    state["handle"] = B.Pool(layers=layers, page_size=page, subs=[(B.HC_TOKEN_ROWS, 2 * e) for e in subs],
                             device_slots=slots, host_pages=0,
                             device_layers=[[t[i] for i in range(layers)] for t in buffers], host=None,
                             stream=torch.cuda.current_stream())
    return B


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(0.0, scale, generator=g)

    def shuffled(n):
        return torch.randperm(n, generator=g, device="cuda")

    state = dict(case=case)
    if case["op"] == "store":
        n, hq, hk, d, dv, slots = (case[k] for k in ("tokens", "q_heads", "kv_heads", "head", "value", "slots"))
        subs = [hk * d] + ([hk * dv] if dv else [])
        state.update(pool=[normal(2, slots, e) for e in subs], q=normal(n, hq, d), k=normal(n, hk, d),
                     v=normal(n, hk, dv) if dv else None, q_out=torch.empty((n, hq, d), dtype=dt, device="cuda"),
                     positions=torch.randint(0, case["far"], (n,), generator=g, device="cuda"),
                     slots=shuffled(slots)[:n].contiguous())
        if own:
            B = _pool(state, subs, 2, slots, case["page"])
            scale = dict(none={}, linear=dict(factor=case["factor"]),
                         llama3=dict(factor=case["factor"], original_context=case["original"]),
                         yarn=dict(factor=case["factor"], original_context=case["original"]))[case["scaling"]]
            state["rope"] = B.Rope(rot_dim=case["rot"], base=case["base"], interleaved=case["interleaved"],
                                   rot_offset=case["rot_offset"], scaling=case["scaling"], **scale)
        return state
    if case["op"] == "attend":
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
        subs = [hk * d] + ([] if d == 576 else [hk * dv])
        state.update(pool=[normal(2, pages * page, e) for e in subs], table=table, kv_len=kv_len,
                     q=normal(sum(q), hq, d, scale=2.0),
                     q_start=torch.tensor([0] + q, device="cuda").cumsum(0),
                     out=torch.empty((sum(q), hq, dv), dtype=dt, device="cuda"))
        if own:
            _pool(state, subs, 2, pages * page, page)
        return state
    layers, page, row, pages = (case[k] for k in ("layers", "page", "row", "pages"))
    ragged = _spread(case["parents"] if case["op"] == "fork" else case["sequences"], case["kv_len"], True)
    lens = torch.tensor(ragged, device="cuda")[shuffled(len(ragged))]
    width = -(-case["kv_len"] // page)
    live = torch.arange(width, device="cuda")[None, :] < ((lens + page - 1) // page)[:, None]
    place = shuffled(pages)
    count = int(live.sum())
    table = torch.full((len(ragged), width), -1, dtype=torch.int64, device="cuda")
    table[live] = place[:count]
    state.update(pool=[normal(layers, pages * page, row // 2) for _ in range(2)], table=table, lens=lens)
    if case["op"] == "fork":
        n = case["children"]
        # every prompt is branched equally often, in any order
        state.update(parents=(torch.arange(n, device="cuda") % len(ragged))[shuffled(n)],
                     free=place[count:].contiguous(), out=torch.empty((n, width), dtype=torch.int64, device="cuda"))
    else:
        state.update(out=torch.empty_like(table))
    if own:
        _pool(state, [row // 2] * 2, layers, pages * page, page)
    return state


# ---------------------------------------------------------------- plain forms
def _frequencies(case):
    """Radians per position of each rotated pair, and the factor on sines and cosines."""
    n = case["rot"] // 2
    i = torch.arange(n, dtype=torch.float64, device="cuda")
    f = torch.exp(-math.log(case["base"]) * i / n)
    if case["scaling"] == "linear":
        return f / case["factor"], 1.0
    if case["scaling"] == "llama3":
        turns = case["original"] * f / (2 * math.pi)  # over the original context; kept above 4, divided below 1
        keep = ((turns - 1.0) / 3.0).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / case["factor"]), 1.0
    if case["scaling"] == "yarn":
        def dim(t):
            return n * math.log(case["original"] / (t * 2 * math.pi)) / math.log(case["base"])
        low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), 2 * n - 1)
        keep = 1 - ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / case["factor"]), 0.1 * math.log(case["factor"]) + 1.0
    return f, 1.0


def _rotated(case, x, positions):
    f, magnitude = _frequencies(case)
    angle = positions.double()[:, None] * f  # 64 bits: far positions
    cos, sin = (angle.cos() * magnitude).float()[:, None], (angle.sin() * magnitude).float()[:, None]
    a, r = case["rot_offset"], case["rot"]
    part = x[..., a:a + r].float()
    if case["interleaved"]:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1).flatten(-2)
    else:
        x1, x2 = part[..., : r // 2], part[..., r // 2:]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)
    return torch.cat([x[..., :a].float(), turned, x[..., a + r:].float()], dim=-1).to(x.dtype)


def _plain_store(s):
    case, slots = s["case"], s["slots"]
    s["q_out"].copy_(_rotated(case, s["q"], s["positions"]))
    s["pool"][0][1].index_copy_(0, slots, _rotated(case, s["k"], s["positions"]).flatten(1))
    if s["v"] is not None:
        s["pool"][1][1].index_copy_(0, slots, s["v"].flatten(1))


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
    k = s["pool"][0][1].view(-1, hk, d)[slot].float().permute(0, 2, 3, 1).contiguous()  # b hk d n
    q = q.view(b, m, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)  # b hk (group m) d
    score = torch.matmul(q, k).view(b, hk, hq // hk, m, n).mul_(d ** -0.5)
    seen = _visible(case, position[:, :, None], key) & there[:, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = score.sum(-1, keepdim=True)
    del k
    v = s["pool"][0][1].view(-1, hk, d)[slot][..., :dv] if d == 576 else s["pool"][1][1].view(-1, hk, dv)[slot]
    v = v.float().permute(0, 2, 1, 3).contiguous()
    out = torch.matmul(score.view(b, hk, -1, n), v).view(b, hk, hq // hk, m, dv)
    out = (out / torch.where(total == 0, 1.0, total)).permute(0, 3, 1, 2, 4).reshape(b, m, hq, dv)
    s["out"].copy_(out[seq, at].to(s["out"].dtype))
    if not case["lse"]:
        return None
    return (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(b, m, hq)[seq, at]


def _plain_fork(s):
    case, parent = s["case"], s["parents"]
    p = case["page"]
    length = s["lens"][parent]
    column = torch.arange(s["table"].shape[1], device="cuda")[None]
    part = length % p > 0
    last = length // p
    own_page = s["free"][(part.cumsum(0) - 1).clamp(min=0)]
    old = s["table"][parent]
    fresh = (column == last[:, None]) & part[:, None]
    table = torch.where(fresh, own_page[:, None], torch.where(column < last[:, None], old, -1))
    s["out"].copy_(table)
    # the filled rows of every partly filled page, one list of slots
    row = torch.arange(p, device="cuda")[None]
    chosen = (row < (length % p)[:, None])
    source = (old.gather(1, last.clamp(max=old.shape[1] - 1)[:, None]) * p + row)[chosen]
    target = (own_page[:, None] * p + row)[chosen]
    for t in s["pool"]:
        t[:, target] = t[:, source]
    return part.sum()[None]


def _plain_compact(s):
    case, p = s["case"], s["case"]["page"]
    n = case["pages"]
    page = torch.arange(n, device="cuda")
    column = torch.arange(s["table"].shape[1], device="cuda")[None]
    entry = column < ((s["lens"] + p - 1) // p)[:, None]
    live = torch.zeros(n + 1, dtype=torch.bool, device="cuda")
    live[torch.where(entry, s["table"], n)] = True
    live = live[:n]
    count = live.sum()
    source = page[live & (page >= count)]
    target = page[~live & (page < count)]
    moved = page.clone()
    moved[source] = target
    s["out"].copy_(torch.where(entry, moved[s["table"].clamp(min=0)], s["table"]))
    for t in s["pool"]:
        v = t.view(case["layers"], n, -1)
        v[:, target] = v[:, source]
    return count[None]


# ---------------------------------------------------------------- one call
def run(state):
    case = state["case"]
    if case["op"] == "store":
        if own:
            state["handle"].store_tokens(1, state["slots"], state["k"], state["v"], q=state["q"], q_out=state["q_out"],
                                         rope=state["rope"], positions=state["positions"])
        else:
            _plain_store(state)
        return {"q": state["q_out"], "pool": state["pool"]}
    if case["op"] == "attend":
        if own:
            lse = state["handle"].attend(1, state["q"], state["table"], state["kv_len"], q_start=state["q_start"],
                                         kv_heads=case["kv_heads"], max_q=case["q_len"], max_kv=case["kv_len"],
                                         entry_tokens=case["entry"], causal=case["causal"], window=case["window"],
                                         sinks=case["sinks"], out=state["out"], return_lse=case["lse"])[1]
        else:
            lse = _plain_attend(state)
        return {"out": state["out"], "lse": lse} if case["lse"] else {"out": state["out"]}
    if case["op"] == "fork":
        if own:
            used = state["handle"].fork_pages(state["table"], state["lens"], state["parents"], state["free"], state["out"])
        else:
            used = _plain_fork(state)
    elif own:
        used = state["handle"].compact_pages(state["table"], state["lens"], state["out"])
    else:
        used = _plain_compact(state)
    return {"table": state["out"], "count": used, "pool": state["pool"]}


# ---------------------------------------------------------------- the definitions, in 64 bits
def _exact_angles(case, positions):
    pairs = case["rot"] // 2
    theta = []
    for i in range(pairs):
        f = case["base"] ** (-2.0 * i / case["rot"])
        wave = 2 * math.pi / f
        if case["scaling"] == "linear":
            f /= case["factor"]
        elif case["scaling"] == "llama3":
            if wave > case["original"]:
                f /= case["factor"]
            elif wave > case["original"] / 4:
                smooth = (case["original"] / wave - 1) / 3
                f = (1 - smooth) * f / case["factor"] + smooth * f
        elif case["scaling"] == "yarn":
            def index(beta):
                return case["rot"] * math.log(case["original"] / (beta * 2 * math.pi)) / (2 * math.log(case["base"]))
            lo, hi = max(math.floor(index(32)), 0), min(math.ceil(index(1)), case["rot"] - 1)
            ramp = min(max((i - lo) / ((hi - lo) or 0.001), 0.0), 1.0)
            f = f / case["factor"] * ramp + f * (1 - ramp)
        theta.append(f)
    magnitude = 0.1 * math.log(case["factor"]) + 1 if case["scaling"] == "yarn" else 1.0
    return positions.double()[:, None] * torch.tensor(theta, dtype=torch.float64, device="cuda"), magnitude


def _exact_turn(case, x, positions):
    angle, magnitude = _exact_angles(case, positions)
    z = torch.polar(torch.full_like(angle, magnitude), angle)[:, None]
    y = x.double().clone()
    a, h = case["rot_offset"], case["rot"] // 2
    first = slice(a, a + 2 * h, 2) if case["interleaved"] else slice(a, a + h)
    second = slice(a + 1, a + 2 * h, 2) if case["interleaved"] else slice(a + h, a + 2 * h)
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        pool = [t.double() for t in s["pool"]]
        pool[0][1, s["slots"]] = _exact_turn(case, s["k"], s["positions"]).flatten(1)
        if s["v"] is not None:
            pool[1][1, s["slots"]] = s["v"].double().flatten(1)
        return {"q": _exact_turn(case, s["q"], s["positions"]), "pool": pool}
    if case["op"] == "attend":
        hk, d, dv, e = (case[k] for k in ("kv_heads", "head", "value", "entry"))
        group = case["q_heads"] // hk
        out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["out"].shape[:2], dtype=torch.float64, device="cuda")
        start, lens = s["q_start"].tolist(), s["kv_len"].tolist()
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            rows = s["table"][b][j // e] * e + j % e
            for h in range(hk):
                k = s["pool"][0][1][rows, h * d:(h + 1) * d].double()
                v = k[:, :dv] if d == 576 else s["pool"][1][1][rows, h * dv:(h + 1) * dv].double()
                kt = k.t().contiguous()
                for r in range(start[b], start[b + 1], 1024):
                    stop = min(r + 1024, start[b + 1])
                    p = n - (start[b + 1] - torch.arange(r, stop, device="cuda"))[:, None, None]
                    x = torch.matmul(s["q"][r:stop, h * group:(h + 1) * group].double(), kt) / math.sqrt(d)
                    if case["causal"]:
                        hidden = j > p
                        if case["window"]:
                            hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
                        x = x.masked_fill(hidden, -math.inf)
                    out[r:stop, h * group:(h + 1) * group] = torch.matmul(torch.softmax(x, -1), v)
                    lse[r:stop, h * group:(h + 1) * group] = torch.logsumexp(x, -1)
        return {"out": out, "lse": lse} if case["lse"] else {"out": out}
    # copies: whole numbers, and payload that moves bit for bit
    p = case["page"]
    table, lens, pool = s["table"].tolist(), s["lens"].tolist(), [t.double() for t in s["pool"]]
    if case["op"] == "fork":
        free, rows, used = s["free"].tolist(), [], 0
        before = [t.clone() for t in pool]
        for r in s["parents"].tolist():
            full, rest = divmod(lens[r], p)
            row = table[r][:full]
            if rest:
                new, old = free[used], table[r][full]
                used += 1
                row = row + [new]
                for t, u in zip(pool, before):
                    t[:, new * p:new * p + rest] = u[:, old * p:old * p + rest]
            rows.append(row + [-1] * (len(table[r]) - len(row)))
        return {"table": torch.tensor(rows), "count": torch.tensor([used]), "pool": pool}
    named = sorted({x for row, n in zip(table, lens) for x in row[:-(-n // p)]})
    count = len(named)
    holes = [x for x in range(count) if x not in set(named)] if count < case["pages"] else []
    to = dict(zip([x for x in named if x >= count], holes))
    before = [t.clone() for t in pool]
    for x, y in to.items():
        for t, u in zip(pool, before):
            t[:, y * p:(y + 1) * p] = u[:, x * p:(x + 1) * p]
    rows = [[to.get(x, x) if j < -(-n // p) else x for j, x in enumerate(row)] for row, n in zip(table, lens)]
    return {"table": torch.tensor(rows), "count": torch.tensor([count]), "pool": pool}
