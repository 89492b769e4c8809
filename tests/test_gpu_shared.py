"""Decode attention for batches that share prefixes."""
import pytest
import torch

import gqa_attention_kv_gb300 as gq
import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")
DTYPE = {"bf16": gq.ATTN_KV_BF16, "fp8": gq.ATTN_KV_FP8_E4M3,
         "e4m3": gq.ATTN_KV_FP8_E4M3_SCALED, "int8": gq.ATTN_KV_INT8_SCALED}
# Weights rounded to f16 (2^-11) and the shared part's normalised sums once more (2^-11)
BITS = 10


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Case:
    """prefix: (row, length) of every request.  Slots that hold no visible key are NaN (or
    the codes of it; INT8: random codes)."""

    def __init__(self, fmt, kind, prefix, tails, R, Hq, H, D, per, seed, window=0,
                 head_major=False, sb=16, more_rows=0, hole=True):
        g = gen(seed)
        self.fmt, self.kind, self.R, self.window, self.H, self.D = fmt, kind, R, window, H, D
        B = len(prefix)
        rows = B + more_rows
        self.prows = torch.tensor([p[0] for p in prefix], dtype=torch.int32)
        self.plens = torch.tensor([p[1] for p in prefix], dtype=torch.int32)
        self.lens = self.plens + torch.tensor(tails, dtype=torch.int32)
        self.pos = (self.lens[:, None] - R + torch.arange(R)).reshape(-1).int()
        longest = int(self.lens.max())
        self.longest, self.max_prefix = longest, max(1, int(self.plens.max()))
        self.table = None
        if kind == gq.PAGED:
            width = -(-longest // per)
            pages = rows * width + 2
            self.table = torch.randperm(pages, generator=g)[:rows * width].view(rows, width).int()
            slots = pages * per
        else:
            per = -(-longest // per) * per
            slots = rows * per
        self.per = per
        used = torch.zeros(slots, dtype=torch.bool)
        for b in range(B):
            for t in range(int(self.lens[b])):
                used[self.slot(b, t)] = True
        if fmt == "bf16":
            k, v = (torch.randn(slots, H, D, generator=g).bfloat16() for _ in range(2))
            odd = NAN
        elif fmt == "int8":
            k, v = (torch.randint(-127, 128, (slots, H, D), generator=g).to(torch.int8)
                    for _ in range(2))
            odd = -128
        else:
            one = torch.tensor(1.0, dtype=torch.float64)
            k, v = (ref.encode("e4m3", torch.randn(slots, H, D, generator=g).double() *
                               (1 if fmt == "fp8" else 60), one) for _ in range(2))
            odd = 0x7F
        if hole:
            k[~used], v[~used] = odd, odd
        if hole and kind == gq.PAGED:  # pages that only hold other rows' prefixes are not there
            for b in range(rows):
                for j in range(self.table.shape[1]):
                    lo = j * per
                    if not used[int(self.table[b, j]) * per:(int(self.table[b, j]) + 1) * per].any():
                        self.table[b, j] = -1
        scaled = fmt in ("e4m3", "int8")
        more = {}
        self.kd, self.vd = k.double() if fmt == "bf16" else None, None
        if fmt == "bf16":
            self.kd, self.vd = k.double(), v.double()
        elif scaled:
            ks, vs = (torch.rand(slots // sb, H, generator=g) * 0.02 + 0.01 for _ in range(2))
            self.kd, self.vd = (ref.dequantized(fmt, x, s, sb) for x, s in ((k, ks), (v, vs)))
            more = dict(k_scale=ks.to(DEV), v_scale=vs.to(DEV), scale_block=sb)
        else:
            self.kd, self.vd = (ref.code_values("e4m3", x) for x in (k, v))
        lay = lambda x: x if not head_major else \
            x.view(-1, per, H, D).transpose(1, 2).contiguous()  # noqa: E731
        self.q = torch.randn(B, R, Hq, D, generator=g).bfloat16()
        self.cache = gq.KVCache(
            kind, lay(k).to(DEV), lay(v).to(DEV), slots_per_seq=0 if kind == gq.PAGED else per,
            block_table=None if self.table is None else self.table.to(DEV),
            block_size=per if kind == gq.PAGED else 0, dtype=DTYPE[fmt],
            layout=gq.ATTN_LAYOUT_BHSD if head_major else gq.ATTN_LAYOUT_BSHD, **more)

    def slot(self, b, t):
        row = int(self.prows[b]) if t < int(self.plens[b]) else b
        if self.kind == gq.PAGED:
            return int(self.table[row, t // self.per]) * self.per + t % self.per
        return row * self.per + t

    def want(self, scale=None):
        return ref.decode(self.q, self.kd, self.vd, self.slot, self.lens, self.pos, self.window, 0,
                          scale or self.D ** -0.5)

    def run(self, scale=None, err=None, **kw):
        args = [x.to(DEV) for x in (self.lens, self.pos, self.prows, self.plens)]
        return gq.attn_decode_shared(self.q.to(DEV), self.cache, *args, self.longest,
                                     self.max_prefix, self.window, scale or self.D ** -0.5,
                                     err=err, **kw)

    def check(self, scale=None, bits=BITS):
        want, mass = self.want(scale)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = self.run(scale, err)
        assert int(err) == 0
        ref.check_output(got, want, mass, weight_bits=bits)
        assert torch.equal(got, self.run(scale))  # timing does not show
        return got


def one_group(n, p):
    return [(0, p)] * n


@pytest.mark.parametrize("fmt,kind,prefix,tails,R,Hq,H,D,per,window,head_major", [
    # one request, one key of its own behind one shared
    ("bf16", gq.LINEAR, one_group(1, 1), [1], 1, 4, 1, 128, 1, 0, False),
    ("bf16", gq.LINEAR, one_group(2, 130), [1, 20], 1, 8, 2, 128, 16, 0, False),
    ("bf16", gq.LINEAR, one_group(5, 700), [3, 40, 17, 3, 90], 3, 14, 2, 64, 8, 0, True),
    # rows of more than one tile, and of more than two
    ("bf16", gq.PAGED, one_group(40, 300), list(range(1, 41)), 1, 16, 4, 128, 16, 0, False),
    ("bf16", gq.PAGED, one_group(75, 140), list(range(4, 79)), 4, 2, 2, 64, 16, 0, True),
    # pages of odd sizes, of one token, larger than a tile
    ("bf16", gq.PAGED, one_group(4, 333), [5, 1, 60, 9], 1, 7, 1, 128, 5, 0, False),
    ("bf16", gq.PAGED, one_group(3, 97), [5, 1, 60], 1, 6, 2, 64, 24, 0, True),
    ("bf16", gq.PAGED, one_group(3, 60), [5, 1, 20], 1, 4, 2, 64, 1, 0, False),
    ("bf16", gq.PAGED, one_group(3, 400), [5, 1, 20], 1, 4, 2, 128, 192, 0, False),
    # heads that are not shared, and many that are
    ("bf16", gq.LINEAR, one_group(9, 260), list(range(1, 10)), 1, 5, 5, 64, 1, 0, False),
    ("bf16", gq.LINEAR, one_group(3, 260), [1, 2, 3], 2, 130, 2, 64, 1, 0, False),
    ("bf16", gq.LINEAR, one_group(2, 200), [1, 2], 1, 128, 1, 128, 1, 0, False),
    # several groups, requests without a prefix between them, one member
    ("bf16", gq.PAGED, [(0, 200)] * 3 + [(3, 0)] + [(4, 500)] * 4 + [(8, 0)] + [(9, 77)],
     [3, 9, 200, 50, 1, 2, 3, 4, 700, 8], 1, 8, 2, 128, 16, 0, False),
    # one row's prefix at two lengths; a group cut in two by another
    ("bf16", gq.LINEAR, [(0, 300)] * 3 + [(0, 150)] * 2 + [(0, 300)] * 2,
     [5, 6, 7, 30, 3, 4, 5], 2, 4, 2, 128, 4, 0, False),
    # nothing shared at all
    ("bf16", gq.LINEAR, [(0, 0), (1, 0)], [40, 300], 1, 8, 2, 128, 16, 0, False),
    # windows that end in the own keys, in the prefix, on its last key
    ("bf16", gq.LINEAR, one_group(4, 300), [50, 60, 100, 200], 1, 8, 2, 128, 16, 40, False),
    ("bf16", gq.PAGED, one_group(4, 500), [50, 60, 100, 20], 3, 8, 2, 64, 16, 111, False),
    ("bf16", gq.PAGED, one_group(3, 500), [11, 12, 13], 1, 8, 2, 64, 16, 13, False),
    # 8-bit caches
    ("e4m3", gq.LINEAR, one_group(6, 500), [5, 6, 7, 30, 3, 64], 1, 8, 2, 128, 16, 0, False),
    ("int8", gq.LINEAR, one_group(6, 500), [5, 6, 7, 30, 3, 64], 2, 8, 2, 64, 16, 0, True),
    ("int8", gq.PAGED, one_group(40, 300), list(range(1, 41)), 1, 16, 2, 128, 16, 0, False),
    ("e4m3", gq.PAGED, [(0, 200)] * 3 + [(3, 0)] + [(4, 500)] * 4, [3, 9, 20, 50, 1, 2, 3, 4], 1,
     12, 2, 64, 32, 90, True),
    ("fp8", gq.LINEAR, one_group(5, 333), [5, 6, 7, 30, 3], 1, 8, 2, 128, 1, 0, False),
    ("fp8", gq.PAGED, one_group(5, 140), [5, 6, 7, 30, 3], 3, 8, 2, 128, 5, 0, False),
    ("fp8", gq.PAGED, one_group(20, 600), list(range(1, 21)), 1, 28, 4, 128, 16, 0, True),
])
def test_shared(fmt, kind, prefix, tails, R, Hq, H, D, per, window, head_major):
    tails = [max(t, R) for t in tails]
    Case(fmt, kind, prefix, tails, R, Hq, H, D, per, len(tails) + D + per, window,
         head_major).check()


@pytest.mark.parametrize("sb,per", [(32, 32), (64, 128), (128, 128)])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_long_scale_blocks(fmt, sb, per):
    Case(fmt, gq.PAGED, one_group(5, 300), [4, 5, 6, 7, 8], 1, 8, 2, 128, per, sb, sb=sb).check()


def test_prefix_in_a_row_outside_the_batch():
    """A text kept in a table row of its own."""
    Case("bf16", gq.PAGED, [(6, 260)] * 6, [1, 2, 3, 4, 5, 6], 1, 8, 2, 128, 16, 3,
         more_rows=1).check()
    Case("bf16", gq.LINEAR, [(4, 260)] * 3, [1, 2, 3], 1, 8, 2, 64, 16, 3, more_rows=2).check()


def test_agrees_with_decode_over_forked_tables():
    """Forked rows name the leader's pages: attn_decode reads the same keys."""
    c = Case("bf16", gq.PAGED, one_group(6, 256), [5, 9, 30, 1, 2, 3], 1, 8, 2, 128, 16, 21)
    got = c.check()
    c.cache.k.nan_to_num_(0.0), c.cache.v.nan_to_num_(0.0)
    c.cache.block_table[:, :16] = c.cache.block_table[0, :16].clone()
    plain = gq.attn_decode(c.q.to(DEV), c.cache, c.lens.to(DEV), c.pos.to(DEV), c.longest, 0,
                           128 ** -0.5)
    want, mass = c.want()
    ref.check_output(plain, want, mass, weight_bits=11)
    ref.check_output(got, want, mass, weight_bits=BITS)


@pytest.mark.parametrize("fmt", ["bf16", "int8"])
def test_rows_without_keys_and_short_lengths(fmt):
    """Lengths that end inside the prefix, at 0, rows at their own positions."""
    c = Case(fmt, gq.LINEAR, one_group(6, 300), [4] * 6, 2, 8, 2, 128, 16, 5, hole=False)
    c.lens = torch.tensor([0, 1, 150, 300, 301, 304], dtype=torch.int32)
    c.pos = torch.tensor([5, -1, 0, 400, 149, 20, 299, 100, -7, 300, 303, 302], dtype=torch.int32)
    got = c.check()
    assert not got[0].any() and not got[4, 0].any()


def test_positions_far_below_zero():
    """They attend nothing, wherever the key tiles lie; a window beside them may be any int32."""
    c = Case("bf16", gq.LINEAR, one_group(5, 300), [4] * 5, 2, 8, 2, 128, 16, 6)
    low = -2 ** 31
    c.pos = torch.tensor([low, 303, 302, low + 1, -2, low + 299, 302, 303, 300, low], dtype=torch.int32)
    for window in (0, 2 ** 31 - 1, 20):
        c.window = window
        got = c.check()
        assert not got[0, 0].any() and not got[1, 1].any() and not got[2].any()


def test_own_slots_before_the_prefix_are_not_read():
    """... nor anything behind a request's last key; table entries there are -1."""
    c = Case("bf16", gq.PAGED, one_group(3, 96), [1, 40, 2], 1, 8, 2, 128, 16, 5)
    assert (c.table[1:, :6] == -1).all() and (c.table[0, 7:] == -1).all()
    c.check()


@pytest.mark.parametrize("D", [64, 128])
def test_late_maxima_and_small_weights(D):
    """Scores that grow along the prefix (the maximum moves late, by jumps), and one heavy
    key beside many light ones."""
    c = Case("bf16", gq.LINEAR, one_group(40, 1000), list(range(1, 41)), 1, 4, 1, D, 8, 9,
             hole=False)
    c.q[:] = 0
    c.q[..., 0] = 1
    ramp = torch.zeros(c.kd.shape[0])
    t = torch.arange(1000)
    for kind in ("ramp", "jumps", "heavy"):
        ramp[:1000] = {"ramp": t / 40.0, "jumps": (t // 130) * 6.0,
                       "heavy": (t == 400) * 9.0}[kind]
        c.kd[:, 0, 0] = ramp.bfloat16().double()
        c.cache.k.copy_(c.kd.bfloat16().to(DEV))
        c.check(scale=1.0)


def test_values_that_are_not_finite():
    """Behind the prefix's end and in masked places they reach nothing; shared ones without
    an f16 are reported."""
    c = Case("bf16", gq.LINEAR, one_group(3, 200), [5, 6, 7], 1, 8, 2, 128, 16, 5)
    c.check()  # NaN everywhere else already
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    base = c.run()
    for bad in (float("inf"), NAN, 70000.0):
        c.cache.v[:300] = torch.where(c.cache.v[:300].isfinite(), c.cache.v[:300], 0)
        keep = c.cache.v[17].clone()
        c.cache.v[17, 0, 3] = bad
        err.zero_()
        out = c.run(err=err)
        assert int(err) == gq.ATTN_ERR_UNSUPPORTED
        assert torch.isfinite(out).all() and torch.equal(out[:, :, 4:], base[:, :, 4:])
        c.cache.v[17] = keep
    # a key that is not finite makes its heads' rows NaN, not the others
    c.cache.k[17, 0, 0] = NAN
    out = c.run()
    assert torch.isnan(out[:, :, :4]).all() and torch.equal(out[:, :, 4:], base[:, :, 4:])


def test_reports():
    c = Case("bf16", gq.PAGED, one_group(3, 200), [5, 6, 7], 1, 8, 2, 128, 16, 5)
    good = c.run()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def reported(change):
        saved = c.prows.clone(), c.plens.clone(), c.lens.clone(), c.cache.block_table.clone()
        change()
        err.zero_()
        out = c.run(err=err)
        torch.cuda.synchronize()
        c.prows, c.plens, c.lens = saved[:3]
        c.cache.block_table.copy_(saved[3])
        return int(err), out

    def row(value):
        c.prows[1] = value

    for value in (-1, 3, 2 ** 31 - 1, -2 ** 31):
        rc, out = reported(lambda: row(value))
        assert rc == gq.ATTN_ERR_BOUNDS and torch.equal(out[[0, 2]], good[[0, 2]])
        assert torch.isfinite(out).all()

    def length(value):  # (its own slots before the prefix's end are NaN)
        c.plens[2] = value

    for value in (-1, 201, 2 ** 31 - 1, -2 ** 31):
        assert reported(lambda: length(value))[0] == gq.ATTN_ERR_BOUNDS

    def page(value):
        c.cache.block_table[0, 3] = value

    for value in (-1, 10 ** 6, -2 ** 31):
        rc, out = reported(lambda: page(value))
        assert rc == gq.ATTN_ERR_BOUNDS and torch.isfinite(out).all()

    def lens(value):
        c.lens[0] = value

    for value in (-1, c.longest + 1, 2 ** 31 - 1):
        assert reported(lambda: lens(value))[0] == gq.ATTN_ERR_BOUNDS
    # unread: the row of a request without a prefix
    c.plens[1], c.prows[1] = 0, 99
    c.lens[1] = 0
    err.zero_()
    c.run(err=err)
    assert int(err) == 0


def test_stream_graph_and_one_workspace():
    c = Case("bf16", gq.PAGED, one_group(20, 300), list(range(1, 21)), 1, 8, 2, 128, 16, 5)
    need = gq.attn_decode_shared_workspace_size(c.cache, 20, 1, 8, c.longest, c.max_prefix)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    out, want = torch.empty_like(c.q, device=DEV), c.run()
    q, lens, pos, prows, plens = (x.to(DEV) for x in (c.q, c.lens, c.pos, c.prows, c.plens))

    def call(stream=None):
        gq.attn_decode_shared(q, c.cache, lens, pos, prows, plens, c.longest, c.max_prefix, 0,
                              128 ** -0.5, out=out, workspace=ws, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    # groups, lengths and positions are read by the replay
    for new_plens in ([300] * 20, [0] * 20, [300] * 7 + [160] * 13, [0, 300] * 10):
        c.plens = torch.tensor(new_plens, dtype=torch.int32)
        c.prows = torch.zeros(20, dtype=torch.int32)
        # requests that share nothing attend their few own keys only
        c.lens = torch.where(c.plens > 0, c.plens, 0) + torch.arange(1, 21).int()
        c.lens = torch.where(c.plens == 160, 160, c.lens)
        c.lens = torch.where(c.plens == 0, 0, c.lens)
        c.pos = c.lens - 1
        plens.copy_(c.plens), prows.copy_(c.prows), lens.copy_(c.lens), pos.copy_(c.pos)
        graph.replay()
        exact, mass = c.want()
        ref.check_output(out, exact, mass, weight_bits=BITS)
    # attn_decode and the window with sinks take the same workspace
    flat = Case("bf16", gq.LINEAR, [(0, 0), (1, 0)], [200, 100], 1, 8, 2, 128, 16, 3)
    a = [x.to(DEV) for x in (flat.lens, flat.pos)]
    big = torch.zeros(max(need, gq.attn_decode_workspace_size(flat.cache, 2, 1, 8, 200)),
                      dtype=torch.uint8, device=DEV)
    exact, mass = flat.want()
    flat.cache.k.nan_to_num_(0.0), flat.cache.v.nan_to_num_(0.0)
    for _ in range(2):
        gq.attn_decode_shared(q, c.cache, lens, pos, prows, plens, c.longest, c.max_prefix, 0,
                              128 ** -0.5, workspace=big)
        ref.check_output(gq.attn_decode(flat.q.to(DEV), flat.cache, *a, 200, 0, 128 ** -0.5,
                                        workspace=big), exact, mass, weight_bits=11)


def test_two_calls_at_once():
    """On two streams, eager and as graphs, each with its workspace."""
    cases = [Case("bf16", gq.PAGED, one_group(30, 900), list(range(1, 31)), 1, 8, 2, 128, 16, 7),
             Case("int8", gq.LINEAR, one_group(9, 2000), list(range(1, 10)), 2, 16, 4, 64, 16, 8)]
    calls, wants, outs, streams, graphs = [], [], [], [], []
    for c in cases:
        wants.append(c.run())
        need = gq.attn_decode_shared_workspace_size(c.cache, c.q.shape[0], c.R, c.q.shape[2],
                                                    c.longest, c.max_prefix)
        ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
        outs.append(torch.empty_like(wants[-1]))
        on = [x.to(DEV) for x in (c.lens, c.pos, c.prows, c.plens)]
        calls.append(lambda c=c, q=c.q.to(DEV), on=on, out=outs[-1], ws=ws: gq.attn_decode_shared(
            q, c.cache, *on, c.longest, c.max_prefix, 0, c.D ** -0.5, out=out, workspace=ws))
        streams.append(torch.cuda.Stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            calls[-1]()
    torch.cuda.synchronize()
    for go in (calls, [g.replay for g in graphs]):
        for out in outs:
            out.fill_(NAN)
        torch.cuda.synchronize()
        for _ in range(5):
            for s, f in zip(streams, go):
                with torch.cuda.stream(s):
                    f()
        torch.cuda.synchronize()
        for out, want in zip(outs, wants):
            assert torch.equal(out, want)


def test_many_requests():
    """Past the tables of one launch, groups of every size."""
    prefix, first = [], 0
    for size in (1, 2, 3, 50, 100, 1, 144):
        prefix += [(first, 20 + 9 * (size % 5))] * size
        first += size
    tails = [1 + i % 7 for i in range(len(prefix))]
    Case("bf16", gq.PAGED, prefix, tails, 1, 4, 2, 64, 8, 30).check()


@pytest.mark.parametrize("fmt,D,G,kind", [("bf16", 64, 1, gq.PAGED), ("int8", 64, 2, gq.LINEAR),
                                          ("bf16", 128, 70, gq.LINEAR), ("e4m3", 128, 3, gq.PAGED)])
def test_more_units_than_sms(fmt, D, G, kind):
    """Forty groups of eight KV heads: a CTA works on one piece after another, tiles full and
    alone in turn, rows of a tile that hold no query."""
    prefix, first = [], 0
    for i in range(40):
        size = (1, 2, 5)[i % 3]
        prefix += [(first, 17 + 31 * (i % 7))] * size
        first += size
    tails = [1 + i % 5 for i in range(first)]
    H = 8 if G < 70 else 5
    Case(fmt, kind, prefix, tails, 1, G * H, H, D, 16, 40 + D + G).check()


def test_own_keys_of_many_requests_in_two_launches():
    """Past 256 (request, row block) pairs, each with own keys of several chunks."""
    n = 300
    c = Case("bf16", gq.LINEAR, one_group(n, 40), [1 + (7 * i) % 90 for i in range(n)], 1, 2, 1, 64,
             8, 77)
    c.check()
    c = Case("int8", gq.LINEAR, one_group(150, 40), [40 + i % 50 for i in range(150)], 20, 2, 2, 64,
             16, 78)  # two blocks of rows a request
    c.check()


def test_a_long_prefix_and_offsets_past_32_bits():
    """Slots whose bytes lie past 2^32 from the cache's start, keys in constant stretches:
    the answer is known."""
    H, D, n = 8, 128, 40000
    rows = (1 << 31) // (H * D * n) + 2
    v = torch.zeros(rows * n, H, D, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(rows * n, H, D, dtype=torch.bfloat16, device=DEV)
    lead = rows - 1
    v[lead * n:lead * n + 30000] = 1.0
    v[lead * n + 15000:lead * n + 30000] = 3.0
    cache = gq.KVCache(gq.LINEAR, k, v, slots_per_seq=n)
    B = 3
    q = torch.randn(B, 1, 16, D, generator=gen(1)).bfloat16().to(DEV)
    lens = torch.tensor([30001, 30002, 30003], dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    out = gq.attn_decode_shared(q, cache, lens, lens - 1, torch.full((B,), lead, **i32),
                                torch.full((B,), 30000, **i32), n, 30000, 0, 0.1)
    # equal scores: the mean, 2 less its own keys' share (zeros)
    want = 60000.0 / lens.double()
    assert ((out.double() - want[:, None, None, None]).abs() <= 2 * (2.0 ** -8 + 2.0 ** -10)).all()


def test_tensors_are_refused():
    c = Case("bf16", gq.PAGED, one_group(3, 64), [1, 2, 3], 1, 8, 2, 128, 16, 5)
    q, lens, pos, prows, plens = (x.to(DEV) for x in (c.q, c.lens, c.pos, c.prows, c.plens))

    def no(q=q, lens=lens, pos=pos, prows=prows, plens=plens, longest=c.longest, most=64, window=0,
           scale=0.1, cache=c.cache, **kw):
        with pytest.raises(gq.AttnError):
            gq.attn_decode_shared(q, cache, lens, pos, prows, plens, longest, most, window, scale,
                                  **kw)

    no(q=q.float())
    no(q=q.cpu())
    no(prows=prows.long())
    no(plens=plens.cpu())
    no(plens=plens[:2])
    no(prows=torch.zeros(6, dtype=torch.int32, device=DEV)[::2])
    no(lens=lens.long())
    no(most=-1)
    no(scale=0.0)
    no(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    no(out=q.float())
    ring = gq.KVCache(gq.RING, c.cache.k, c.cache.v, slots_per_seq=100)
    no(cache=ring, window=50)
