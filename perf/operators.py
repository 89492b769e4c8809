"""The operators around the KV cache as they are measured: attention over an
8-bit cache with a scale per block of tokens and head, attention with a sliding
window and sinks, and the page operations of a paged cache.

``run`` computes a pass either in plain torch operations (``own`` false) or
through this package's entry points (``own`` true).
"""
import math

import torch

own = False

DEV = "cuda"
SCALE_FLOOR = 2.0 ** -64
QMAX = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's new token of 64 requests into a paged 8-bit cache
        {"name": "append8 step", "op": "append8", "fmt": "e4m3", "kind": "paged", "batch": 64,
         "rows": 1, "hkv": 8, "hd": 128, "lo": 64, "hi": 1024, "block": 16, "sblock": 16},
        # a whole prompt's rows into a fresh linear 8-bit cache
        {"name": "append8 prompt", "op": "append8", "fmt": "e4m3", "kind": "linear", "batch": 1,
         "rows": 14449, "hkv": 4, "hd": 128, "lo": 14449, "hi": 14449, "block": 0, "sblock": 16},
        # the smallest decode: one request, one row, 512 keys (latency)
        {"name": "decode8 one", "op": "decode8", "fmt": "e4m3", "kind": "linear", "batch": 1,
         "rows": 1, "hq": 32, "hkv": 8, "hd": 128, "lo": 512, "hi": 512, "block": 0, "sblock": 16},
        # several rows a request over a paged pool, ragged lengths
        {"name": "decode8 paged", "op": "decode8", "fmt": "int8", "kind": "paged", "batch": 64,
         "rows": 4, "hq": 32, "hkv": 8, "hd": 128, "lo": 64, "hi": 4096, "block": 16,
         "sblock": 16},
        # few requests at long contexts, seven query heads to a KV head
        {"name": "decode8 long", "op": "decode8", "fmt": "e4m3", "kind": "linear", "batch": 2,
         "rows": 1, "hq": 28, "hkv": 4, "hd": 128, "lo": 14449, "hi": 23971, "block": 0,
         "sblock": 64},
        # a batch without head sharing, 64-wide heads
        {"name": "decode8 heads", "op": "decode8", "fmt": "int8", "kind": "paged", "batch": 16,
         "rows": 1, "hq": 32, "hkv": 32, "hd": 64, "lo": 2048, "hi": 8192, "block": 64,
         "sblock": 32},
        # speech encoder: 1,500 frames, window 750
        {"name": "prefill sinks encoder", "op": "sink_prefill", "batch": 1, "len": 1500,
         "hq": 32, "hkv": 32, "hd": 64, "window": 750, "sinks": 4},
        # a long prompt under a sliding window
        {"name": "prefill sinks prompt", "op": "sink_prefill", "batch": 1, "len": 14449,
         "hq": 28, "hkv": 4, "hd": 128, "window": 4096, "sinks": 64},
        # one request far past its window, the pages between sinks and window freed (latency)
        {"name": "decode sinks one", "op": "sink_decode", "kind": "paged", "batch": 1, "rows": 1,
         "hq": 32, "hkv": 8, "hd": 128, "lo": 9000, "hi": 9000, "block": 16, "window": 1024,
         "sinks": 4},
        # endless generation over rings that keep their first tokens
        {"name": "decode sinks ring", "op": "sink_decode", "kind": "ring", "batch": 16, "rows": 1,
         "hq": 32, "hkv": 8, "hd": 128, "lo": 8192, "hi": 40000, "block": 16384, "window": 8192,
         "sinks": 4},
        # a beam step: the losing rows' pages are released, the winners' tables forked
        {"name": "pages fork", "op": "fork", "batch": 16, "width": 3, "layers": 26, "hkv": 8,
         "hd": 128, "lo": 200, "hi": 1500, "block": 16},
        # a half-empty pool of 8,192 pages pulled together
        {"name": "pages compact", "op": "compact", "batch": 48, "pages": 8192, "layers": 4,
         "hkv": 8, "hd": 128, "lo": 300, "hi": 2400, "block": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _drawn(rng):
    op = rng.choice(["append8", "decode8", "decode8", "sink_prefill", "sink_decode", "fork",
                     "compact"])
    hd = rng.choice([64, 128])
    if op == "append8":
        kind = rng.choice(["linear", "paged"])
        sblock = rng.choice([16, 32, 64])
        rows = rng.choice([1, rng.randint(2, 9), _log(rng, 10, 4000)])
        batch = _log(rng, 1, max(1, min(128, 16000 // rows)))
        hi = rows + rng.randint(0, 700)
        return {"op": op, "fmt": rng.choice(["e4m3", "int8"]), "kind": kind, "batch": batch,
                "rows": rows, "hkv": rng.choice([1, 2, 4, 8]), "hd": hd, "lo": rows, "hi": hi,
                "block": sblock * rng.choice([1, 2]) if kind == "paged" else 0, "sblock": sblock}
    if op in ("decode8", "sink_decode"):
        hkv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8])
        rows = rng.choice([1, 1, 2, 3, 4, 5])
        batch = _log(rng, 1, 64)
        hi = _log(rng, max(rows, 16), 20000 if batch < 8 else 6000)
        lo = max(rows, hi // rng.choice([1, 2, 20]))
        case = {"op": op, "batch": batch, "rows": rows, "hq": hkv * group, "hkv": hkv, "hd": hd,
                "lo": lo, "hi": hi}
        if op == "decode8":
            kind, sblock = rng.choice(["linear", "paged"]), rng.choice([16, 32, 64])
            return dict(case, fmt=rng.choice(["e4m3", "int8"]), kind=kind, sblock=sblock,
                        block=sblock * rng.choice([1, 2]) if kind == "paged" else 0)
        kind = rng.choice(["linear", "paged", "ring"])
        window, sinks = _log(rng, 8, 8192), _log(rng, 1, 130)
        block = {"linear": 0, "paged": rng.choice([5, 16, 24, 64]),
                 "ring": sinks + window + rows - 1 + rng.randint(0, 300)}[kind]
        return dict(case, kind=kind, block=block, window=window, sinks=sinks)
    if op == "sink_prefill":
        hkv, group = rng.choice([1, 2, 4]), rng.choice([1, 2, 4, 7])
        batch = rng.choice([1, 1, 2, 3])
        n = _log(rng, 64, 9000)
        return {"op": op, "batch": batch, "len": n, "hq": hkv * group, "hkv": hkv, "hd": hd,
                "window": _log(rng, 16, max(17, n)), "sinks": _log(rng, 1, 300)}
    case = {"op": op, "hkv": rng.choice([1, 2, 4, 8]), "hd": hd, "block": rng.choice([16, 32, 24])}
    if op == "fork":
        hi = _log(rng, 20, 3000)
        return dict(case, batch=_log(rng, 1, 24), width=rng.randint(1, 4),
                    layers=rng.randint(1, 28), lo=max(1, hi // 8), hi=hi)
    hi = _log(rng, 50, 3000)
    batch = _log(rng, 4, 64)
    pages = int(batch * (hi // case["block"] + 1) * rng.uniform(1.3, 2.5)) + 16
    return dict(case, batch=batch, pages=pages, layers=rng.randint(1, 4), lo=max(1, hi // 8),
                hi=hi)


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = {c["op"] == "sink_prefill": _cost(c) for c in sorted(listed(), key=_cost)}
    while True:
        case = _drawn(rng)
        if _cost(case) <= most[case["op"] == "sink_prefill"]:
            return case


# ------------------------------------------------------------------- the work
def _lengths(case):
    """Tokens of each request: spread evenly over lo .. hi."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi if b == 1 else lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _seen(n, window, sinks):
    """Keys that the row at position n - 1 sees."""
    return n if n <= window + sinks else window + sinks


def work(case):
    op = case["op"]
    if op == "append8":
        n, row = case["batch"] * case["rows"], case["hkv"] * case["hd"]
        scales = 2 * 4 * case["hkv"] * (n // case["sblock"] + case["batch"])
        return {"bytes": n * row * 2 * 3 + 8 * n + scales, "flops": 4 * n * row}
    if op in ("decode8", "sink_decode"):
        esize = 1 if op == "decode8" else 2
        keys = 0
        for n in _lengths(case):
            keys += n if op == "decode8" else min(n, _seen(n, case["window"], case["sinks"]) +
                                                  case["rows"] - 1)
        qrows = case["batch"] * case["rows"] * case["hq"]
        scales = 2 * 4 * case["hkv"] * (keys // case["sblock"]) if op == "decode8" else 0
        return {"bytes": 2 * keys * case["hkv"] * case["hd"] * esize + scales +
                4 * qrows * case["hd"], "flops": 4 * keys * case["rows"] * case["hq"] * case["hd"]}
    if op == "sink_prefill":
        n, w, s = case["len"], case["window"], case["sinks"]
        full = min(n, w + s)  # rows that see every key up to their own
        pairs = full * (full + 1) // 2 + (n - full) * (w + s)
        return {"bytes": 2 * case["batch"] * n * case["hd"] * 2 * (case["hq"] + case["hkv"]),
                "flops": 4 * case["batch"] * case["hq"] * pairs * case["hd"]}
    bs, row = case["block"], case["hkv"] * case["hd"] * 2
    if op == "fork":
        kids = case["width"]
        part = sum(n % bs for n in _lengths(case)) * kids
        entries = sum(-(-n // bs) for n in _lengths(case)) * (1 + kids)
        return {"bytes": case["layers"] * part * row * 2 * 2 + 4 * 2 * entries, "flops": 0}
    used = sum(-(-n // bs) for n in _lengths(case)) - case["lo"] // bs // 2 * (case["batch"] // 2)
    moved = used * max(0.0, 1.0 - used / case["pages"])
    return {"bytes": case["layers"] * moved * bs * row * 2 * 2 + 4 * 2 * (used + case["pages"]),
            "flops": 0}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _codes(g, fmt, *shape):
    """Codes as N(0, 1) rows leave them: the largest of a block near the end of the range."""
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float16)
    if fmt == "int8":
        return (x * 36).round_().clamp_(-127, 127).to(torch.int8)
    return (x * 125).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(g, fmt, *shape):
    return (3.2 + 0.9 * torch.rand(*shape, generator=g, device=DEV)) / QMAX[fmt]


def _lens(g, case):
    n = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    return n[torch.randperm(len(n), generator=g, device=DEV)]


def _table(g, lens, bs, pool=None):
    """A table whose pages are dealt from a shuffled pool; -1 past a request's last page."""
    b, width = len(lens), int(-(-int(lens.max()) // bs))
    col = torch.arange(width, device=DEV)
    has = col[None, :] < -(-lens[:, None] // bs)
    pool = pool or int(has.sum()) + 7
    table = torch.full((b, width), -1, dtype=torch.int32, device=DEV)
    table[has] = torch.randperm(pool, generator=g, device=DEV)[: int(has.sum())].int()
    return table, pool


def _slots(state, t):
    """Cache slots of positions t [batch, n] (any value where the table holds no page)."""
    case, t = state["case"], t.long()
    rows = torch.arange(t.shape[0], device=DEV)[:, None]
    if case["kind"] == "paged":
        bs = case["block"]
        return state["table"].long()[rows, t // bs].clamp(min=0) * bs + t % bs
    per = state["per_seq"]
    if case["kind"] == "ring":
        s = case["sinks"]
        t = torch.where(t < s, t, s + (t - s) % (per - s))
    return rows * per + t


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    st = {"case": dict(case), "table": None, "per_seq": 0}
    if op == "sink_prefill":
        b, n, hd = case["batch"], case["len"], case["hd"]
        st.update(q=_bf16(g, b, n, case["hq"], hd), k=_bf16(g, b, n, case["hkv"], hd),
                  v=_bf16(g, b, n, case["hkv"], hd), scale=hd ** -0.5)
        return st
    if op in ("fork", "compact"):
        return _prepare_pages(st, case, g)
    b, r, hkv, hd = case["batch"], case["rows"], case["hkv"], case["hd"]
    lens = _lens(g, case)
    st["lens"] = lens
    if case["kind"] == "paged":
        st["table"], pages = _table(g, lens, case["block"])
        slots = pages * case["block"]
    else:
        step = case.get("sblock", 1)
        st["per_seq"] = case["block"] or -(-int(lens.max()) // step) * step
        slots = b * st["per_seq"]
    if op == "sink_decode":
        st["k"], st["v"] = _bf16(g, slots, hkv, hd), _bf16(g, slots, hkv, hd)
    else:
        fmt, blocks = case["fmt"], slots // case["sblock"]
        st["k"], st["v"] = _codes(g, fmt, slots, hkv, hd), _codes(g, fmt, slots, hkv, hd)
        st["ks"], st["vs"] = _scales(g, fmt, blocks, hkv), _scales(g, fmt, blocks, hkv)
    pos = lens[:, None] - r + torch.arange(r, device=DEV, dtype=torch.int32)
    if op == "append8":
        st.update(k_new=_bf16(g, b * r, hkv, hd), v_new=_bf16(g, b * r, hkv, hd),
                  slots=_slots(st, pos).reshape(-1))
        st["touched"] = torch.unique(st["slots"] // case["sblock"])
        return st
    st.update(q=_bf16(g, b, r, case["hq"], hd), pos=pos.reshape(-1).contiguous(),
              scale=hd ** -0.5)
    if op == "sink_decode" and case["kind"] == "paged":
        # pages wholly between the sinks and the oldest row's window have been given back
        col = torch.arange(st["table"].shape[1], device=DEV) * case["block"]
        gone = (col >= case["sinks"]) & (col[None, :] + case["block"] <=
                                         (lens[:, None] - r + 1 - case["window"]))
        st["table"][gone] = -1
    return st


def _prepare_pages(st, case, g):
    b, bs, lens = case["batch"], case["block"], _lens(g, case)
    need = int((-(-lens // bs)).sum())
    if case["op"] == "fork":
        kids = b * case["width"]
        parents, pages = _table(g, lens, bs, need + 2 * kids + need // 4)
        table = torch.full((b + kids, parents.shape[1]), -1, dtype=torch.int32, device=DEV)
        table[:b] = parents
        src = torch.arange(b, device=DEV, dtype=torch.int32).repeat_interleave(case["width"])
        st.update(src=src, dst=torch.arange(b, b + kids, device=DEV, dtype=torch.int32),
                  fork_lens=lens[src.long()].contiguous(),
                  zero=torch.zeros(kids, dtype=torch.int32, device=DEV),
                  ends=torch.full((kids,), table.shape[1], dtype=torch.int32, device=DEV))
        most = kids
    else:
        pages = case["pages"]
        table, _ = _table(g, lens, bs, pages)
        # every other request shares its neighbour's first half
        half = int(lens.min()) // bs // 2
        table[1:2 * (b // 2):2, :half] = table[0:2 * (b // 2):2, :half]
        st["case_table"] = table.clone()
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs.index_put_((table[table >= 0].long(),), torch.ones((), dtype=torch.int32, device=DEV),
                    accumulate=True)
    if case["op"] == "compact":
        # room for the moves that a pool filled at random needs, and some more
        used = need - half * (b // 2)
        expected = used * (1 - used / pages)
        most = min(int(expected + 5 * math.sqrt(expected)) + 8, pages - used)
        assert used == int((refs > 0).sum()) and int((refs[used:] > 0).sum()) <= most
        st["case_refs"] = refs.clone()
        st["used"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    shape = (case["layers"], pages * bs, case["hkv"], case["hd"])
    st.update(table=table, refs=refs, k=_bf16(g, *shape), v=_bf16(g, *shape),
              moves=torch.zeros(most, 3, dtype=torch.int32, device=DEV),
              n_moves=torch.zeros(1, dtype=torch.int32, device=DEV))
    return st


# --------------------------------------------------------------- a whole pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"append8": _own_append8, "decode8": _own_decode8, "sink_decode": _own_sink_decode,
                "sink_prefill": _own_sink_prefill, "fork": _own_fork,
                "compact": _own_compact}[op](state)
    return {"append8": _append8, "decode8": _decode8, "sink_decode": _sink_decode,
            "sink_prefill": _sink_prefill, "fork": _fork, "compact": _compact}[op](state)


def _append_out(st):
    """The cache after the call: the values of its codes, and its scales."""
    if st["case"]["fmt"] == "e4m3":
        k, v = st["k"].view(torch.float8_e4m3fn), st["v"].view(torch.float8_e4m3fn)
    else:
        n = st["case"]["sblock"]
        k = (st["k"].view(-1, n, *st["k"].shape[1:]) * st["ks"][:, None, :, None])
        v = (st["v"].view(-1, n, *st["v"].shape[1:]) * st["vs"][:, None, :, None])
    return {"k": k, "v": v, "ks": st["ks"], "vs": st["vs"]}


# ------------------------------------------------ this package's entry points
def _cache(st):
    import gqa_attention_kv_gb300 as gq

    if "cache" not in st:
        case = st["case"]
        kind = {"linear": gq.LINEAR, "paged": gq.PAGED, "ring": gq.RING}[case["kind"]]
        more = {}
        if "fmt" in case:
            more = dict(dtype={"e4m3": gq.ATTN_KV_FP8_E4M3_SCALED,
                               "int8": gq.ATTN_KV_INT8_SCALED}[case["fmt"]],
                        k_scale=st["ks"], v_scale=st["vs"], scale_block=case["sblock"])
        paged = case["kind"] == "paged"
        st["cache"] = gq.KVCache(kind, st["k"], st["v"], slots_per_seq=st["per_seq"],
                                 block_table=st["table"] if paged else None,
                                 block_size=case["block"] if paged else 0, **more)
    return gq, st["cache"]


def _own_append8(st):
    gq, cache = _cache(st)
    gq.attn_kv_append(st["k_new"], st["v_new"], st["slots"], cache)
    return _append_out(st)


def _own_decode8(st):
    gq, cache = _cache(st)
    case = st["case"]
    if "ws" not in st:
        need = gq.attn_decode_workspace_size(cache, case["batch"], case["rows"], case["hq"],
                                             case["hi"])
        st["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return gq.attn_decode(st["q"], cache, st["lens"], st["pos"], case["hi"], 0, st["scale"],
                          workspace=st["ws"])


def _own_sink_decode(st):
    gq, cache = _cache(st)
    case = st["case"]
    if "ws" not in st:
        need = gq.attn_decode_sinks_workspace_size(cache, case["batch"], case["rows"], case["hq"],
                                                   case["hi"], case["window"], case["sinks"])
        st["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    return gq.attn_decode_sinks(st["q"], cache, st["lens"], st["pos"], case["hi"], case["window"],
                                case["sinks"], st["scale"], workspace=st["ws"])


def _own_sink_prefill(st):
    import gqa_attention_kv_gb300 as gq

    return gq.attn_prefill_sinks(st["q"], st["k"], st["v"], st["case"]["window"],
                                 st["case"]["sinks"], st["scale"])


def _own_copy(gq, st):
    if "caches" not in st:
        bs = st["case"]["block"]
        st["caches"] = [gq.KVCache(gq.PAGED, st["k"][i], st["v"][i], block_table=st["table"],
                                   block_size=bs) for i in range(st["case"]["layers"])]
    gq.attn_pages_copy(st["caches"], st["moves"], st["n_moves"])


def _own_fork(st):
    import gqa_attention_kv_gb300 as gq

    gq.attn_pages_free(st["table"], st["refs"], st["dst"], st["zero"], st["ends"])
    gq.attn_pages_fork(st["table"], st["refs"], st["src"], st["dst"], st["fork_lens"],
                       st["case"]["block"], st["moves"], st["n_moves"])
    _own_copy(gq, st)
    return _pages_out(st)


def _own_compact(st):
    import gqa_attention_kv_gb300 as gq

    # the pool as it stood before the call (its pages' data is still in place)
    st["table"].copy_(st["case_table"])
    st["refs"].copy_(st["case_refs"])
    if "ws" not in st:
        need = gq.attn_pages_workspace_size(st["refs"].shape[0])
        st["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    gq.attn_pages_compact(st["table"], st["refs"], st["case"]["block"], st["moves"],
                          st["n_moves"], st["used"], workspace=st["ws"])
    _own_copy(gq, st)
    return _pages_out(st)


def _pages_out(st):
    out = {"table": st["table"], "refs": st["refs"], "moves": st["moves"],
           "n_moves": st["n_moves"], "k": st["k"], "v": st["v"]}
    if "used" in st:
        out["used"] = st["used"]
    return out


# ------------------------------------------------------------- the plain form
def _decode_codes(fmt, c):
    return c.float() if fmt == "int8" else c.view(torch.float8_e4m3fn).float()


def _encode(fmt, x, by):
    """Codes of x * by (both in 32 bits).  INT8 rounds the exact product, formed
    in 64 bits: half a maximum lies on the border of two codes."""
    if fmt == "int8":
        return (x.double() * by.double()).round().clamp(-127, 127).to(torch.int8)
    return (x * by).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _append8_one(st, codes, scale, new):
    """One tensor (K or V): the touched blocks' scales grow to hold the new
    rows, their earlier codes follow, then the rows are encoded.  A block whose
    first slot is written starts anew."""
    fmt, sb = st["case"]["fmt"], st["case"]["sblock"]
    hkv, hd = codes.shape[1:]
    slots, touched = st["slots"], st["touched"]
    x, block = new.float(), slots // sb
    first = torch.zeros(scale.shape[0], dtype=torch.int32, device=DEV)
    first.index_add_(0, block, (slots % sb == 0).int())
    held = torch.where((first > 0)[:, None], SCALE_FLOOR, scale)
    amax = torch.zeros_like(scale)
    amax.scatter_reduce_(0, block[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    now = torch.maximum(held, amax / torch.full_like(amax, QMAX[fmt]))
    inv = torch.ones_like(now) / now
    blocks = codes.view(-1, sb, hkv, hd)
    was = blocks[touched]
    again = _encode(fmt, _decode_codes(fmt, was),
                    (scale * inv)[touched][:, None, :, None])
    grown = (first[touched][:, None] == 0) & (now[touched] > scale[touched])
    blocks[touched] = torch.where(grown[:, None, :, None], again, was)
    codes[slots] = _encode(fmt, x, inv[block][:, :, None])
    scale[touched] = now[touched]


def _append8(st):
    _append8_one(st, st["k"], st["ks"], st["k_new"])
    _append8_one(st, st["v"], st["vs"], st["v_new"])
    return _append_out(st)


def _attend(q, k, v, see, scale):
    """q [b, r, hq, d]; k, v [b, t, hkv, d] in 32 bits; see [b, r, t]."""
    b, r, hq, d = q.shape
    hkv = k.shape[2]
    q = q.float().view(b, r, hkv, hq // hkv, d)
    s = torch.einsum("brhgd,bthd->bhrgt", q, k) * scale
    s.masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True).clamp_(min=-1e30)
    s.sub_(top).exp_()
    total = s.sum(-1)
    o = torch.einsum("bhrgt,bthd->bhrgd", s, v) / total.clamp(min=1e-30)[..., None]
    return o.permute(0, 2, 1, 3, 4).reshape(b, r, hq, d).to(torch.bfloat16)


def _decode8(st):
    case = st["case"]
    t = torch.arange(case["hi"], device=DEV, dtype=torch.int32).expand(case["batch"], -1)
    if case["kind"] == "paged":
        t = t.clamp(max=st["table"].shape[1] * case["block"] - 1)
    slots = _slots(st, t)
    block = slots // case["sblock"]
    k = _decode_codes(case["fmt"], st["k"][slots]) * st["ks"][block][..., None]
    v = _decode_codes(case["fmt"], st["v"][slots]) * st["vs"][block][..., None]
    pos = st["pos"].view(case["batch"], case["rows"], 1)
    see = (t[:, None, :] <= pos) & (t[:, None, :] < st["lens"][:, None, None])
    return _attend(st["q"], k, v, see, st["scale"])


def _sink_decode(st):
    case, lens = st["case"], st["lens"]
    s, w, r = case["sinks"], case["window"], case["rows"]
    # the sinks, then the positions that some row's window reaches
    span = min(case["hi"], w + r - 1)
    sink = torch.arange(min(s, case["hi"]), device=DEV, dtype=torch.int32)
    near = lens[:, None] - span + torch.arange(span, device=DEV, dtype=torch.int32)
    t = torch.cat([sink.expand(case["batch"], -1), near], 1)
    real = torch.cat([sink[None, :] < lens[:, None], near >= s], 1)
    slots = _slots(st, torch.where(real, t, 0))
    k, v = st["k"][slots].float(), st["v"][slots].float()
    pos = st["pos"].view(case["batch"], r, 1)
    t = t[:, None, :]
    see = real[:, None, :] & (t <= pos) & ((t < s) | (pos - t < w))
    return _attend(st["q"], k, v, see, st["scale"])


def _sink_prefill(st):
    case = st["case"]
    b, n, hq, d = st["q"].shape
    group = hq // case["hkv"]
    q = st["q"].float().permute(0, 2, 1, 3).reshape(b, case["hkv"], group * n, d)
    k = st["k"].float().permute(0, 2, 3, 1)
    v = st["v"].float().permute(0, 2, 1, 3)
    s = torch.matmul(q * st["scale"], k).view(b, hq, n, n)
    i = torch.arange(n, device=DEV)
    gap = i[:, None] - i[None, :]
    see = (gap >= 0) & ((gap < case["window"]) | (i[None, :] < case["sinks"]))
    s.masked_fill_(~see, -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(b, case["hkv"], group * n, n), v).view(b, hq, n, d) / total
    return o.permute(0, 2, 1, 3).to(torch.bfloat16)


def _in_order(wanted, size):
    """Indices of the true entries of `wanted`, ascending, in the first places
    of a list of `size` (the rest: len(wanted))."""
    n = wanted.shape[0]
    place = torch.where(wanted, wanted.cumsum(0) - 1, size).clamp(max=size)
    got = torch.full((size + 1,), n, dtype=torch.int64, device=DEV)
    got[place] = torch.where(wanted, torch.arange(n, device=DEV), n)
    return got[:size]


def _copy_pages(st, src, dst, rows):
    """Rows 0 .. rows - 1 of page src[i] to page dst[i], in every layer."""
    bs = st["case"]["block"]
    take = (torch.arange(bs, device=DEV) < rows[:, None])[None, :, :, None, None]
    k = st["k"].view(st["k"].shape[0], -1, bs, *st["k"].shape[2:])
    v = st["v"].view(k.shape)
    k[:, dst] = torch.where(take, k[:, src], k[:, dst])
    v[:, dst] = torch.where(take, v[:, src], v[:, dst])


def _fork(st):
    bs, table, refs = st["case"]["block"], st["table"], st["refs"]
    src, dst, lens = st["src"].long(), st["dst"].long(), st["fork_lens"].long()
    pages, kids = refs.shape[0], src.shape[0]
    # the old rows' pages lose a reference each
    old = table[dst].long()
    refs.index_add_(0, old.clamp(min=0).reshape(-1), -(old >= 0).int().reshape(-1))
    # full pages are shared; a partial last page is copied to the lowest free one
    col = torch.arange(table.shape[1], device=DEV)[None, :]
    row = table[src].long()
    full, part = (lens // bs)[:, None], lens % bs
    shared = torch.where(col < full, row, -1)
    free = _in_order(refs == 0, 2 * kids)
    refs.index_add_(0, shared.clamp(min=0).reshape(-1), (shared >= 0).int().reshape(-1))
    some = part > 0
    order = some.long().cumsum(0) - 1
    moved = some.long().sum()
    spare = free[moved + (~some).long().cumsum(0) - 1]  # stands in where nothing is copied
    new = torch.where(some, free[order.clamp(min=0)], spare)
    last = row.gather(1, full.clamp(max=table.shape[1] - 1))[:, 0]
    table[dst] = torch.where((col == full) & some[:, None], new[:, None], shared).int()
    refs.index_add_(0, new, some.int())
    triple = torch.stack([last, new, part], 1).int()
    place = _in_order(some, kids).clamp(max=kids - 1)
    listed_ = torch.arange(kids, device=DEV)[:, None] < moved
    st["moves"].copy_(torch.where(listed_, triple[place], st["moves"]))
    st["n_moves"].copy_(moved.int())
    _copy_pages(st, torch.where(some, last, new), new, part)
    return _pages_out(st)


def _compact(st):
    st["table"].copy_(st["case_table"])
    st["refs"].copy_(st["case_refs"])
    table, refs, bs = st["table"], st["refs"], st["case"]["block"]
    pages, most = refs.shape[0], st["moves"].shape[0]
    page = torch.arange(pages, device=DEV)
    used = refs > 0
    n = used.sum()
    leaves, takes = used & (page >= n), ~used & (page < n)
    src, dst = _in_order(leaves, most), _in_order(takes, most)
    moved = leaves.sum()
    real = torch.arange(most, device=DEV) < moved
    spare = _in_order(~used & (page >= n), most)  # stands in where nothing is copied
    spare = spare[(torch.arange(most, device=DEV) - moved).clamp(min=0)]
    src, dst = torch.where(real, src, spare), torch.where(real, dst, spare)
    to = page.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    refs[dst] = refs[src]
    refs.copy_(torch.where(page < n, refs, 0))
    triple = torch.stack([src, dst, torch.full_like(src, bs)], 1).int()
    st["moves"].copy_(torch.where(real[:, None], triple, st["moves"]))
    st["n_moves"].copy_(moved.int())
    st["used"].copy_(n.int())
    _copy_pages(st, src, dst, torch.where(real, bs, 0))
    return _pages_out(st)


# ------------------------------------------------------- what it is, in 64 bits
def exact(case, seed):
    """The definitions, request by request and head by head, in 64 bits.  The
    page operations only move values: there is nothing to compute."""
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    st = prepare(case, seed)
    if op == "append8":
        return _exact_append(st)
    if op == "sink_prefill":
        return _exact_prefill(st)
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    hkv, r = case["hkv"], case["rows"]
    group = case["hq"] // hkv
    for b, n in enumerate(st["lens"].tolist()):
        pos = torch.arange(n - r, n, device=DEV)[:, None]
        t = torch.arange(n, device=DEV)
        see = t[None, :] <= pos
        if op == "sink_decode":
            see &= (pos - t[None, :] < case["window"]) | (t[None, :] < case["sinks"])
            t = t[see.any(0)]
            see = see[:, t]
        if case["kind"] == "paged":
            slot = st["table"][b].long()[t // case["block"]] * case["block"] + t % case["block"]
        elif case["kind"] == "linear":
            slot = b * st["per_seq"] + t
        else:
            turn = st["per_seq"] - case["sinks"]
            slot = b * st["per_seq"] + torch.where(
                t < case["sinks"], t, case["sinks"] + torch.remainder(t - case["sinks"], turn))
        k, v = st["k"][slot], st["v"][slot]
        if op == "decode8":
            if case["fmt"] == "e4m3":
                k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            block = torch.div(slot, case["sblock"], rounding_mode="floor")
            k = k.double() * st["ks"].double()[block].unsqueeze(-1)
            v = v.double() * st["vs"].double()[block].unsqueeze(-1)
        k, v = k.double(), v.double()
        for h in range(hkv):
            qh = st["q"][b, :, h * group:(h + 1) * group].double()  # [r, group, d]
            s = st["scale"] * (qh @ k[:, h].T)
            p = torch.softmax(s.masked_fill(~see[:, None, :], -math.inf), -1)
            out[b, :, h * group:(h + 1) * group] = p @ v[:, h]
    return out


def _exact_prefill(st):
    case = st["case"]
    b, n, hq, d = st["q"].shape
    if b * hq * n * n * d * 4 > 8e12:
        return None
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    i = torch.arange(n, device=DEV)
    hidden = (i[None, :] > i[:, None]) | ((i[:, None] - i[None, :] >= case["window"]) &
                                          (i[None, :] >= case["sinks"]))
    for x in range(b):
        for h in range(hq):
            g = h // (hq // case["hkv"])
            s = st["q"][x, :, h].double() @ st["k"][x, :, g].double().T
            p = torch.softmax(s.mul_(st["scale"]).masked_fill_(hidden, -math.inf), -1)
            out[x, :, h] = p @ st["v"][x, :, g].double()
    return out


def _exact_append(st):
    """Scales are held in 32 bits and so are their reciprocals: both are
    rounded to that, everything else is in 64 bits."""
    case = st["case"]
    sb, top = case["sblock"], QMAX[case["fmt"]]
    int8 = case["fmt"] == "int8"

    def values(c):
        return (c if int8 else c.view(torch.float8_e4m3fn)).double()

    def nearest(x):
        if int8:
            return torch.clamp(torch.round(x), -top, top)
        # E4M3: three fraction bits, the smallest step 2^-9
        x = torch.clamp(x, -top, top)
        e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(e - 3)
        return torch.round(x / step) * step

    def held32(x):
        return x.float().double()

    out = {}
    for name, codes, scale, new in (("k", st["k"], st["ks"], st["k_new"]),
                                    ("v", st["v"], st["vs"], st["v_new"])):
        held, s, x = values(codes), scale.double(), new.double()
        block = torch.div(st["slots"], sb, rounding_mode="floor")
        begun = torch.zeros(s.shape[0], dtype=torch.bool, device=DEV)
        begun[block[st["slots"] % sb == 0]] = True
        most = torch.zeros_like(s).index_reduce_(0, block, x.abs().amax(-1), "amax")
        mine = torch.zeros(s.shape[0], dtype=torch.bool, device=DEV)
        mine[block] = True
        base = torch.where(begun[:, None], torch.full_like(s, SCALE_FLOOR), s)
        after = held32(torch.where(mine[:, None], torch.maximum(base, most / top), s))
        by = held32(1.0 / after)
        grew = mine[:, None] & ~begun[:, None] & (after > s)
        h = held.view(-1, sb, *held.shape[1:])
        h = torch.where(grew[:, None, :, None], nearest(h * held32(s * by)[:, None, :, None]), h)
        h = h.reshape(held.shape).clone()
        h[st["slots"]] = nearest(x * by[block][:, :, None])
        if int8:
            h = h.view(-1, sb, *held.shape[1:]) * after[:, None, :, None]
        out[name], out[name + "s"] = h, after
    return out
