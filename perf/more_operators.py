"""Operators around a serving step as they are measured: rotary positions with
norms of queries and keys (written to the cache in the same pass), decode
attention for batches that share long prefixes, and reading a cache back.

``run`` computes a pass either in plain torch operations (``own`` false) or
through this package's entry points (``own`` true).
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
QMAX = {"e4m3": 448.0, "int8": 127.0}
SCALED = ("e4m3", "int8")


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of 64 requests: norms, rotation, keys and values into a paged cache
        {"name": "rope step", "op": "rope", "n": 64, "hq": 32, "hkv": 8, "hd": 128, "rot": 128,
         "layout": "half", "norm": True, "scaling": 1.0, "far": 1024, "into": "paged",
         "fmt": "bf16", "block": 16},
        # a whole prompt's queries and keys, from the rows of one fused projection
        {"name": "rope prompt", "op": "rope", "n": 14449, "hq": 28, "hkv": 4, "hd": 128,
         "rot": 128, "layout": "half", "norm": False, "scaling": 1.0, "far": 14449,
         "into": "none", "fmt": "bf16", "block": 0},
        # speech frames: a part of each head turns, in pairs, with norms, far positions
        {"name": "rope frames", "op": "rope", "n": 1500, "hq": 32, "hkv": 32, "hd": 64,
         "rot": 32, "layout": "pairs", "norm": True, "scaling": 8.0, "far": 400000,
         "into": "linear", "fmt": "bf16", "block": 0},
        # one token far into a long text, into an E4M3 cache (latency)
        {"name": "rope one", "op": "rope", "n": 1, "hq": 28, "hkv": 4, "hd": 128, "rot": 128,
         "layout": "pairs", "norm": False, "scaling": 8.0, "far": 1000000, "into": "linear",
         "fmt": "fp8", "block": 0},
        # a prompt kept as INT8 read back as the keys and values of a prefill
        {"name": "read prompt", "op": "read", "fmt": "int8", "n": 14449, "hkv": 4, "hd": 128,
         "kind": "linear", "block": 0, "sblock": 64},
        # the pages of some requests, E4M3, out of a pool (latency)
        {"name": "read pages", "op": "read", "fmt": "e4m3", "n": 500, "hkv": 8, "hd": 128,
         "kind": "paged", "block": 16, "sblock": 16},
        # the smallest shared decode: two continuations of one prompt (latency)
        {"name": "shared two", "op": "shared", "fmt": "bf16", "kind": "linear", "batch": 2,
         "groups": 1, "loners": 0, "prefix": 512, "lo": 1, "hi": 20, "rows": 1, "hq": 32,
         "hkv": 8, "hd": 128, "block": 0, "sblock": 0, "window": 0},
        # 64 requests behind one instruction text, as forks of its pages
        {"name": "shared pages", "op": "shared", "fmt": "bf16", "kind": "paged", "batch": 64,
         "groups": 1, "loners": 0, "prefix": 4096, "lo": 64, "hi": 1024, "rows": 1, "hq": 32,
         "hkv": 8, "hd": 128, "block": 16, "sblock": 0, "window": 0},
        # answers sampled from one long prompt, seven query heads to a KV head
        {"name": "shared long", "op": "shared", "fmt": "bf16", "kind": "linear", "batch": 16,
         "groups": 1, "loners": 0, "prefix": 14449, "lo": 1, "hi": 2000, "rows": 1, "hq": 28,
         "hkv": 4, "hd": 128, "block": 0, "sblock": 0, "window": 0},
        # several texts behind one batch, 8-bit pages, and requests that share nothing
        {"name": "shared groups", "op": "shared", "fmt": "e4m3", "kind": "paged", "batch": 123,
         "groups": 4, "loners": 3, "prefix": 8192, "lo": 16, "hi": 700, "rows": 1, "hq": 32,
         "hkv": 8, "hd": 128, "block": 32, "sblock": 32, "window": 0},
        # several rows a request, heads that share nothing, INT8
        {"name": "shared rows", "op": "shared", "fmt": "int8", "kind": "linear", "batch": 32,
         "groups": 1, "loners": 0, "prefix": 2500, "lo": 4, "hi": 300, "rows": 4, "hq": 32,
         "hkv": 32, "hd": 64, "block": 0, "sblock": 64, "window": 0},
        # the largest: 256 requests behind a long text
        {"name": "shared wide", "op": "shared", "fmt": "bf16", "kind": "paged", "batch": 256,
         "groups": 1, "loners": 0, "prefix": 32768, "lo": 32, "hi": 256, "rows": 1, "hq": 32,
         "hkv": 8, "hd": 128, "block": 64, "sblock": 0, "window": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["rope", "rope", "read", "shared", "shared", "shared"])
    hd, hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    if op == "rope":
        into = rng.choice(["none", "linear", "paged"])
        return {"op": op, "n": _log(rng, 1, 14449), "hq": hkv * rng.choice([1, 2, 3, 4, 7, 8]),
                "hkv": hkv, "hd": hd, "rot": rng.choice([hd, hd, hd // 2, hd // 4, 20, 48]),
                "layout": rng.choice(["half", "pairs"]), "norm": rng.choice([True, False]),
                "scaling": rng.choice([1.0, 1.0, 4.0, 32.0]), "far": _log(rng, 14449, 1000000),
                "into": into, "fmt": "fp8" if into != "none" and hd == 128 and
                rng.random() < 0.3 else "bf16",
                "block": rng.choice([5, 16, 24, 64]) if into == "paged" else 0}
    if op == "read":
        kind, sblock = rng.choice(["linear", "paged"]), rng.choice([16, 32, 64, 128])
        return {"op": op, "fmt": rng.choice(["bf16", "e4m3", "int8"] + ["fp8"] * (hd == 128)),
                "n": _log(rng, 1, 14449), "hkv": hkv, "hd": hd, "kind": kind,
                "block": sblock * rng.choice([1, 2]) if kind == "paged" else 0, "sblock": sblock}
    kind, sblock = rng.choice(["linear", "paged"]), rng.choice([16, 32, 64])
    fmt = rng.choice(["bf16", "bf16", "e4m3", "int8"] + ["fp8"] * (hd == 128))
    group, rows = rng.choice([1, 2, 3, 4, 6, 7, 8]), rng.choice([1, 1, 1, 2, 3, 4])
    groups, loners = rng.choice([1, 1, 2, 3, 5]), rng.choice([0, 0, 1, 3])
    batch = groups * _log(rng, 1, 120 // groups) + loners + rng.randint(0, groups - 1)
    hi = _log(rng, rows, 2000)
    block = 0
    if kind == "paged":
        block = sblock * rng.choice([1, 2]) if fmt in SCALED else rng.choice([5, 16, 24, 64])
    return {"op": op, "fmt": fmt, "kind": kind, "batch": batch, "groups": groups,
            "loners": loners, "prefix": _log(rng, 20, 30000), "lo": max(rows, hi // 20),
            "hi": hi, "rows": rows, "hq": hkv * group, "hkv": hkv, "hd": hd, "block": block,
            "sblock": sblock if fmt in SCALED else 0,
            "window": rng.choice([0, 0, 0, _log(rng, 16, 20000)])}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op)
            for op in ("rope", "read", "shared")}
    while True:
        case = _drawn(rng)
        if _cost(case) > most[case["op"]]:
            continue
        # the caches and the plain form's copies of them fit the card
        if case["op"] == "shared" and case["kind"] == "linear" and \
                case["batch"] * (case["prefix"] + case["hi"]) * case["hkv"] * case["hd"] > 3e9:
            continue
        return case


# ------------------------------------------------------------------- the work
def _members(case):
    """(first request, requests, prefix length) of each group; the loners, last in
    the batch, are groups of their own without a prefix."""
    n, out, at = case["batch"] - case["loners"], [], 0
    for g in range(case["groups"]):
        size = n // case["groups"] + (g < n % case["groups"])
        if size:
            out.append((at, size, max(1, case["prefix"] * (case["groups"] - g) // case["groups"])))
        at += size
    return out + [(n + i, 1, 0) for i in range(case["loners"])]


def _tails(case):
    """Tokens of each request behind its prefix: spread evenly over lo .. hi."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _esize(case):
    return 2 if case["fmt"] == "bf16" else 1


def work(case):
    op, d = case["op"], case["hd"]
    if op == "rope":
        n, turned, v = case["n"], case["hq"] + case["hkv"], 0 if case["into"] == "none" else 1
        row = (turned + v * case["hkv"]) * d * 2
        written = (case["hq"] * 2 + case["hkv"] * (1 + v) * _esize(case)) * d
        return {"bytes": n * (row + written + 4 + 8 * v),
                "flops": n * turned * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if op == "read":
        n, row = case["n"], case["hkv"] * d
        scales = 8 * case["hkv"] * (n // case["sblock"]) if case["fmt"] in SCALED else 0
        return {"bytes": 2 * n * row * (_esize(case) + 2) + scales + 8 * n, "flops": 2 * n * row}
    # a window hides what lies further back than it reaches (from the first of the rows)
    members, r = _members(case), case["rows"]
    w = case["window"] or 1 << 30
    mean = sum(_tails(case)) / case["batch"]
    keys = pairs = 0
    for _, size, p in members:
        keys += min(p, max(0, w + r - 1 - case["lo"])) + size * min(mean, w + r - 1)
        pairs += size * r * min(p + mean, w)
    qo = case["batch"] * r * case["hq"] * d * 2 * 2
    return {"bytes": int(2 * keys * case["hkv"] * d * _esize(case)) + qo,
            "flops": int(4 * pairs * case["hq"] * d)}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _stored(g, fmt, *shape):
    """Cache contents: bf16, or codes as N(0, 1) rows leave them."""
    if fmt == "bf16":
        return _bf16(g, *shape)
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float16)
    if fmt == "int8":
        return (x * 36).round_().clamp_(-127, 127).to(torch.int8)
    return (x if fmt == "fp8" else x * 125).clamp_(-448, 448).to(
        torch.float8_e4m3fn).view(torch.uint8)


def _make_cache(st, g, slots):
    case = st["case"]
    fmt, hkv, hd = case["fmt"], case["hkv"], case["hd"]
    st["k"], st["v"] = _stored(g, fmt, slots, hkv, hd), _stored(g, fmt, slots, hkv, hd)
    if fmt in SCALED:
        shape = (slots // case["sblock"], hkv)
        for name in ("ks", "vs"):
            st[name] = (3.2 + 0.9 * torch.rand(*shape, generator=g, device=DEV)) / QMAX[fmt]
    if fmt == "fp8":
        st["ref"] = torch.randn(hkv, hd, generator=g, device=DEV)


def _frequencies(case):
    """Inverse frequencies of base 10,000; with a scaling the slow ones (fewer than one
    turn in 4,096 tokens) are divided by it and the fast ones (more than 32) are not, a
    linear ramp between, and the cosines and sines grow a little with it."""
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    s = case["scaling"]
    if s == 1.0:
        return inv.float().to(DEV), 1.0
    turns = 4096 * inv / (2 * math.pi)
    keep = ((turns - 1) / 31).clamp(0, 1)
    return (inv * keep + inv / s * (1 - keep)).float().to(DEV), 0.1 * math.log(s) + 1


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": dict(case), "table": None, "per_seq": 0}
    return {"rope": _prepare_rope, "read": _prepare_read, "shared": _prepare_shared}[op](st, g)


def _prepare_rope(st, g):
    case = st["case"]
    n, hq, hkv, hd = case["n"], case["hq"], case["hkv"], case["hd"]
    # the rows of one fused projection: q, k and v are views of it
    fused = _bf16(g, n, hq + 2 * hkv, hd)
    st.update(q=fused[:, :hq], k_new=fused[:, hq:hq + hkv], v_new=fused[:, hq + hkv:])
    st["inv"], st["factor"] = _frequencies(case)
    st["qw"] = st["kw"] = None
    if case["norm"]:
        st["qw"] = 1 + 0.1 * torch.randn(hd, generator=g, device=DEV)
        st["kw"] = 1 + 0.1 * torch.randn(hd, generator=g, device=DEV)
    first = torch.randint(0, max(1, case["far"] - n) + 1, (1,), generator=g, device=DEV)
    if n <= 256:  # a step's requests stand anywhere, a prompt's tokens one behind the other
        pos = torch.randint(0, case["far"], (n,), generator=g, device=DEV)
    else:
        pos = first + torch.arange(n, device=DEV)
    st["pos"] = pos.int()
    if case["into"] == "none":
        return st
    slots = n + 37
    if case["into"] == "paged":
        bs = case["block"]
        pages = -(-slots // bs) + 3
        order = torch.randperm(pages, generator=g, device=DEV)
        i = torch.arange(n, device=DEV) + int(bs // 2)
        st["slots"] = order[i // bs] * bs + i % bs
        slots = pages * bs
        st["table"] = order.int()[None, :].contiguous()
    else:
        st["per_seq"] = slots
        st["slots"] = torch.arange(n, device=DEV) + 11
    _make_cache(st, g, slots)
    return st


def _prepare_read(st, g):
    case = st["case"]
    n, sb = case["n"], case["sblock"]
    unit = case["block"] or sb
    blocks = -(-n // unit) + 5
    st["per_seq"] = blocks * unit
    i = torch.arange(n, device=DEV) + unit // 3
    if case["kind"] == "paged":
        order = torch.randperm(blocks, generator=g, device=DEV)
        st["slots"] = order[i // unit] * unit + i % unit
        st["table"] = order.int()[None, :].contiguous()
    else:
        st["slots"] = i
    _make_cache(st, g, blocks * unit)
    return st


def _prepare_shared(st, g):
    case = st["case"]
    b, r, bs = case["batch"], case["rows"], case["block"]
    tails = torch.tensor(_tails(case), dtype=torch.int32, device=DEV)
    tails = tails[torch.randperm(b, generator=g, device=DEV)]
    lead, plen = [], []
    for first, size, p in _members(case):
        lead += [first] * size
        plen += [p] * size
    lead = torch.tensor(lead, device=DEV)
    st["rows_of"], st["plens"] = lead.int(), torch.tensor(plen, dtype=torch.int32, device=DEV)
    st["lens"] = st["plens"] + tails
    st["longest"] = case["hi"] + (case["prefix"] if case["groups"] else 0)
    if case["kind"] == "paged":
        # as forks leave a table: whole pages of the prefix are the leader's
        width = -(-st["longest"] // bs)
        col = torch.arange(width, device=DEV)
        has = col[None, :] < -(-st["lens"][:, None] // bs)
        theirs = (col[None, :] < (st["plens"] // bs)[:, None]) & \
            (lead != torch.arange(b, device=DEV))[:, None]
        mine = has & ~theirs
        pages = int(mine.sum()) + 5
        table = torch.full((b, width), -1, dtype=torch.int32, device=DEV)
        table[mine] = torch.randperm(pages, generator=g, device=DEV)[: int(mine.sum())].int()
        st["table"] = torch.where(theirs, table[lead], table)
        slots = pages * bs
    else:
        step = case["sblock"] or 1
        st["per_seq"] = -(-st["longest"] // step) * step
        slots = b * st["per_seq"]
    _make_cache(st, g, slots)
    pos = st["lens"][:, None] - r + torch.arange(r, device=DEV, dtype=torch.int32)
    st.update(q=_bf16(g, b, r, case["hq"], case["hd"]), pos=pos.reshape(-1).contiguous(),
              scale=case["hd"] ** -0.5)
    return st


# --------------------------------------------------------------- a whole pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "read": _own_read, "shared": _own_shared}[op](state)
    return {"rope": _rope, "read": _read, "shared": _shared}[op](state)


def _codes_out(st, x):
    return x.view(torch.float8_e4m3fn) if st["case"]["fmt"] == "fp8" else x


# ------------------------------------------------ this package's entry points
def _cache(st):
    import gqa_attention_kv_gb300 as gq

    if "cache" not in st:
        case = st["case"]
        paged = st["table"] is not None
        more = {}
        if case["fmt"] in SCALED:
            more = dict(dtype={"e4m3": gq.ATTN_KV_FP8_E4M3_SCALED,
                               "int8": gq.ATTN_KV_INT8_SCALED}[case["fmt"]],
                        k_scale=st["ks"], v_scale=st["vs"], scale_block=case["sblock"])
        elif case["fmt"] == "fp8":
            more = dict(dtype=gq.ATTN_KV_FP8_E4M3, k_ref=st["ref"])
        st["cache"] = gq.KVCache(gq.PAGED if paged else gq.LINEAR, st["k"], st["v"],
                                 slots_per_seq=0 if paged else st["per_seq"],
                                 block_table=st["table"], block_size=case["block"], **more)
    return gq, st["cache"]


def _own_rope(st):
    import gqa_attention_kv_gb300 as gq

    case = st["case"]
    if "rope" not in st:
        layout = {"half": gq.ATTN_ROPE_HALF, "pairs": gq.ATTN_ROPE_PAIRS}[case["layout"]]
        st["rope"] = gq.Rope(st["inv"], layout=layout, factor=st["factor"], q_weight=st["qw"],
                             k_weight=st["kw"], eps=EPS)
    if case["into"] == "none":
        q, k = gq.attn_qk_rope(st["q"], st["k_new"], st["pos"], st["rope"])
        return {"q": q, "k": k}
    gq, cache = _cache(st)
    q = gq.attn_qk_rope_append(st["q"], st["k_new"], st["v_new"], st["pos"], st["slots"], cache,
                               st["rope"])
    return {"q": q, "k": _codes_out(st, st["k"]), "v": _codes_out(st, st["v"])}


def _own_read(st):
    gq, cache = _cache(st)
    return gq.attn_kv_read(st["slots"], cache)


def _own_shared(st):
    gq, cache = _cache(st)
    case = st["case"]
    if "ws" not in st:
        need = gq.attn_decode_shared_workspace_size(cache, case["batch"], case["rows"], case["hq"],
                                                    st["longest"], case["prefix"], case["window"])
        st["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return gq.attn_decode_shared(st["q"], cache, st["lens"], st["pos"], st["rows_of"],
                                 st["plens"], st["longest"], case["prefix"], case["window"],
                                 st["scale"], workspace=st["ws"])


# ------------------------------------------------------------- the plain form
def _values(st, slots, name):
    """K or V ("k", "v") of some slots in 32 bits."""
    case, x = st["case"], st[name][slots]
    if case["fmt"] in ("fp8", "e4m3"):
        x = x.view(torch.float8_e4m3fn)
    x = x.float()
    if case["fmt"] in SCALED:
        x = x * st[name + "s"][slots // case["sblock"]][..., None]
    return x


def _turn(st, x, weight):
    """Norm and rotation of rows x [n, heads, hd], in 32 bits (angles in 64)."""
    case, x = st["case"], x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    a = st["pos"].double()[:, None] * st["inv"].double()
    c = (a.cos().float() * st["factor"])[:, None, :]
    s = (a.sin().float() * st["factor"])[:, None, :]
    rot = case["rot"]
    if case["layout"] == "half":
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
    else:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).to(torch.bfloat16)


def _rope(st):
    case = st["case"]
    q, k = _turn(st, st["q"], st["qw"]), _turn(st, st["k_new"], st["kw"])
    if case["into"] == "none":
        return {"q": q, "k": k}
    v = st["v_new"]
    if case["fmt"] == "fp8":
        k = (k.float() - st["ref"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = v.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    st["k"][st["slots"]] = k
    st["v"][st["slots"]] = v
    return {"q": q, "k": _codes_out(st, st["k"]), "v": _codes_out(st, st["v"])}


def _read(st):
    k, v = _values(st, st["slots"], "k"), _values(st, st["slots"], "v")
    if st["case"]["fmt"] == "fp8":
        k = k + st["ref"]
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _slots_of(st, rows, t):
    """Slots of positions t of requests `rows` (any slot where the table holds no page)."""
    t = t.long()
    if st["case"]["kind"] == "paged":
        bs = st["case"]["block"]
        page = t.div(bs, rounding_mode="floor").clamp(max=st["table"].shape[1] - 1)
        return st["table"].long()[rows, page].clamp(min=0) * bs + t % bs
    return rows * st["per_seq"] + t.clamp(max=st["per_seq"] - 1)


def _shared(st):
    case, outs = st["case"], []
    hkv, hd, r = case["hkv"], case["hd"], case["rows"]
    group, w = case["hq"] // hkv, case["window"]
    for first, size, p in _members(case):
        q = st["q"][first:first + size].float().view(size, r, hkv, group, hd)
        pos = st["pos"].view(-1, r)[first:first + size, :, None]
        lens = st["lens"][first:first + size, None, None]
        own_t = p + torch.arange(case["hi"], device=DEV)
        t = torch.cat([torch.arange(p, device=DEV), own_t])
        see = (t <= pos) & (t < lens)
        if w:
            see &= pos - t < w
        slots = _slots_of(st, torch.full((1,), first, device=DEV), t[:p])
        kp, vp = _values(st, slots, "k"), _values(st, slots, "v")
        rows = torch.arange(first, first + size, device=DEV)[:, None]
        slots = _slots_of(st, rows, own_t[None, :])
        kt, vt = _values(st, slots, "k"), _values(st, slots, "v")
        s = torch.cat([torch.einsum("nrhgd,thd->hnrgt", q, kp),
                       torch.einsum("nrhgd,nthd->hnrgt", q, kt)], -1)
        s.mul_(st["scale"]).masked_fill_(~see[None, :, :, None, :], -math.inf)
        s.sub_(s.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
        total = s.sum(-1).clamp(min=1e-30)[..., None]
        o = torch.einsum("hnrgt,thd->hnrgd", s[..., :p], vp) + \
            torch.einsum("hnrgt,nthd->hnrgd", s[..., p:], vt)
        outs.append((o / total).permute(1, 2, 0, 3, 4).reshape(size, r, case["hq"], hd))
    return torch.cat(outs).to(torch.bfloat16)


# ------------------------------------------------------- what it is, in 64 bits
def _exact_value(st, name, slot):
    fmt = st["case"]["fmt"]
    c = st[name][slot]
    if fmt in ("e4m3", "fp8"):
        c = c.view(torch.float8_e4m3fn)
    c = c.double()
    if fmt in SCALED:
        block = torch.div(slot, st["case"]["sblock"], rounding_mode="floor")
        c = c * st[name + "s"].double()[block].unsqueeze(-1)
    return c


def exact(case, seed):
    """The definitions in 64 bits, row by row or request by request."""
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    if case["op"] == "read":
        k, v = (_exact_value(st, name, st["slots"]) for name in ("k", "v"))
        return (k + st["ref"].double() if case["fmt"] == "fp8" else k), v
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    group = case["hq"] // case["hkv"]
    lead, plen = st["rows_of"].tolist(), st["plens"].tolist()
    for b, n in enumerate(st["lens"].tolist()):
        pos = torch.arange(n - case["rows"], n, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)
        see = t[None, :] <= pos
        if case["window"]:
            see = see & (pos - t[None, :] < case["window"])
        row = torch.where(t < plen[b], lead[b], b)
        if case["kind"] == "paged":
            page = torch.div(t, case["block"], rounding_mode="floor")
            slot = st["table"].long()[row, page] * case["block"] + t % case["block"]
        else:
            slot = row * st["per_seq"] + t
        k, v = (_exact_value(st, name, slot) for name in ("k", "v"))
        for h in range(case["hkv"]):
            qh = st["q"][b, :, h * group:(h + 1) * group].double()  # [rows, group, d]
            s = st["scale"] * (qh @ k[:, h].T)
            p = torch.softmax(s.masked_fill(~see[:, None, :], -math.inf), -1)
            out[b, :, h * group:(h + 1) * group] = p @ v[:, h]
    return out


def _exact_rope(st):
    case = st["case"]
    rot, hd = case["rot"], case["hd"]
    # a rotation of the plane spanned by two dims of a head, as a complex product
    if case["layout"] == "half":
        first = torch.arange(rot // 2, device=DEV)
        second = first + rot // 2
    else:
        first = 2 * torch.arange(rot // 2, device=DEV)
        second = first + 1
    angle = torch.outer(st["pos"].double(), st["inv"].double())
    by = torch.polar(torch.full_like(angle, st["factor"]), angle)

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            size = torch.sqrt((x ** 2).sum(-1, keepdim=True) / hd + EPS)
            x = x / size * weight.double()
        y = x.clone()
        z = torch.complex(x[..., first], x[..., second]) * by[:, None, :]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k, v = turned(st["q"], st["qw"]), turned(st["k_new"], st["kw"]), st["v_new"].double()
    if case["into"] == "none":
        return {"q": q, "k": k}
    out = {"q": q}
    for name, new in (("k", k), ("v", v)):
        held = st[name]
        if case["fmt"] == "fp8":
            held = held.view(torch.float8_e4m3fn)
            if name == "k":
                new = new.to(torch.bfloat16).double() - st["ref"].double()
            # E4M3: three fraction bits, the smallest step 2^-9
            new = new.clamp(-448, 448)
            step = torch.exp2(torch.floor(torch.log2(new.abs().clamp(min=2.0 ** -6))) - 3)
            new = torch.round(new / step) * step
        held = held.double()
        held[st["slots"]] = new
        out[name] = held
    return out
