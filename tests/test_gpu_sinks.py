"""Sliding windows with sinks: decode over every cache kind, and prefill."""
import math

import pytest
import torch

import gqa_attention_kv_gb300 as gq
import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def build(kind, B, R, Hq, H, D, lo, hi, per, window, sinks, seed, head_major=False, evict=True):
    """A bf16 cache whose slots hold NaN wherever no visible key lies."""
    g = gen(seed)
    lens = torch.randint(lo, hi + 1, (B,), generator=g, dtype=torch.int32)
    lens[0], lens[-1] = lo, hi
    pos = (lens[:, None] - R + torch.arange(R)).reshape(-1).int()
    table = None
    if kind == gq.PAGED:
        width = -(-hi // per)
        pages = B * width + 2
        table = torch.randperm(pages, generator=g)[:B * width].view(B, width).int()
        slots = pages * per
        slot = lambda b, t: int(table[b, t // per]) * per + t % per  # noqa: E731
    else:
        per = per or hi
        slots = B * per
        slot = (lambda b, t: b * per + t) if kind == gq.LINEAR else \
            (lambda b, t: ref.ring_slot(b, t, per, sinks))
    k, v = (torch.full((slots, H, D), NAN).bfloat16() for _ in range(2))
    for b in range(B):
        n = int(lens[b])
        first = n - R + 1 - window if window > 0 else 0
        seen = [t for t in range(n) if t < sinks or t >= first]
        if kind == gq.PAGED and evict:
            for j in range(table.shape[1]):
                if not any(t // per == j for t in seen):
                    table[b, j] = -1
        at = [slot(b, t) for t in seen]
        for x in (k, v):
            x[at] = torch.randn(len(at), H, D, generator=g).bfloat16()
    q = torch.randn(B, R, Hq, D, generator=g).bfloat16()
    lay = lambda x: x if not head_major else \
        x.view(-1, per, H, D).transpose(1, 2).contiguous()  # noqa: E731
    cache = gq.KVCache(kind, lay(k).to(DEV), lay(v).to(DEV),
                       slots_per_seq=0 if kind == gq.PAGED else per,
                       block_table=None if table is None else table.to(DEV),
                       block_size=per if kind == gq.PAGED else 0,
                       layout=gq.ATTN_LAYOUT_BHSD if head_major else gq.ATTN_LAYOUT_BSHD)
    return cache, q, k, v, lens, pos, slot


def run(cache, q, lens, pos, hi, window, sinks, scale, err=None, **kw):
    return gq.attn_decode_sinks(q.to(DEV), cache, lens.to(DEV), pos.to(DEV), hi, window, sinks,
                                scale, err=err, **kw)


@pytest.mark.parametrize("kind,B,R,Hq,H,D,lo,hi,per,window,sinks,head_major", [
    (gq.LINEAR, 1, 1, 4, 1, 128, 1, 1, 0, 8, 4, False),            # one token
    (gq.LINEAR, 3, 1, 8, 8, 64, 3, 500, 0, 100, 4, False),
    (gq.LINEAR, 2, 3, 28, 4, 128, 5, 900, 0, 64, 1, True),         # 21 rows: two units
    (gq.LINEAR, 2, 1, 8, 2, 128, 40, 300, 0, 1, 1, False),         # the row itself and one sink
    (gq.LINEAR, 2, 2, 4, 2, 64, 90, 200, 0, 16, 300, False),       # more sinks than tokens
    (gq.LINEAR, 2, 1, 8, 2, 64, 90, 700, 0, 0, 5, False),          # no window
    (gq.LINEAR, 2, 1, 8, 2, 128, 90, 700, 0, 33, 0, False),        # no sinks
    (gq.PAGED, 3, 1, 8, 2, 128, 20, 800, 16, 60, 4, False),
    (gq.PAGED, 3, 4, 8, 2, 64, 20, 640, 5, 70, 7, False),          # pages of 5
    (gq.PAGED, 2, 2, 16, 2, 128, 300, 333, 24, 100, 30, True),     # pages end inside a chunk
    (gq.PAGED, 2, 1, 4, 4, 64, 40, 900, 1, 50, 3, False),          # pages of one token
    (gq.RING, 4, 1, 8, 2, 128, 1, 1000, 80, 64, 4, False),
    (gq.RING, 3, 4, 8, 8, 64, 4, 777, 141, 100, 17, True),
    (gq.RING, 2, 2, 12, 2, 128, 500, 501, 70, 64, 5, False),
    (gq.RING, 2, 1, 8, 2, 64, 60, 400, 50, 50, 0, False),          # the plain ring
])
def test_decode(kind, B, R, Hq, H, D, lo, hi, per, window, sinks, head_major):
    cache, q, k, v, lens, pos, slot = build(kind, B, R, Hq, H, D, lo, hi, per, window, sinks,
                                            B + hi + D, head_major)
    want, mass = ref.decode(q, k.double(), v.double(), slot, lens, pos, window, sinks, D ** -0.5)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run(cache, q, lens, pos, hi, window, sinks, D ** -0.5, err)
    assert int(err) == 0
    ref.check_output(got, want, mass, weight_bits=16)
    assert torch.equal(got, run(cache, q, lens, pos, hi, window, sinks, D ** -0.5))


def test_decode_without_sinks_is_the_plain_window():
    """n_sinks 0 answers attn_decode's question (by another kernel: both within
    the bound of the same reference)."""
    cache, q, k, v, lens, pos, slot = build(gq.LINEAR, 2, 2, 8, 2, 128, 50, 600, 0, 70, 0, 3)
    cache.k.nan_to_num_(0.0)  # attn_decode wants finite values in masked places
    cache.v.nan_to_num_(0.0)
    want, mass = ref.decode(q, k.double(), v.double(), slot, lens, pos, 70, 0, 0.1)
    ref.check_output(run(cache, q, lens, pos, 600, 70, 0, 0.1), want, mass, weight_bits=16)
    old = gq.attn_decode(q.to(DEV), cache, lens.to(DEV), pos.to(DEV), 600, 70, 0.1)
    ref.check_output(old, want, mass, weight_bits=11)


@pytest.mark.parametrize("dtype", ["fp8", "e4m3", "int8"])
def test_decode_of_8_bit_caches(dtype):
    """Sinks over unscaled E4M3 and scaled caches."""
    g = gen(11)
    H, D, n, window, sinks = 2, 128, 400, 90, 6
    fmt = "int8" if dtype == "int8" else "e4m3"
    one = torch.tensor(1.0, dtype=torch.float64)
    k, v = (ref.encode(fmt, torch.randn(n, H, D, generator=g).double() *
                       (1 if dtype == "fp8" else 40), one) for _ in range(2))
    ks, vs = (torch.rand(n // 16, H, generator=g) * 0.02 + 0.01 for _ in range(2))
    more = {}
    if dtype == "fp8":
        ks, vs = torch.ones_like(ks), torch.ones_like(vs)
    else:
        more = dict(k_scale=ks.to(DEV), v_scale=vs.to(DEV), scale_block=16)
    kind = {"fp8": gq.ATTN_KV_FP8_E4M3, "e4m3": gq.ATTN_KV_FP8_E4M3_SCALED,
            "int8": gq.ATTN_KV_INT8_SCALED}[dtype]
    cache = gq.KVCache(gq.LINEAR, k.to(DEV), v.to(DEV), slots_per_seq=n, dtype=kind, **more)
    q = torch.randn(1, 3, 8, D, generator=g).bfloat16()
    lens, pos = torch.tensor([n], dtype=torch.int32), torch.arange(n - 3, n, dtype=torch.int32)
    want, mass = ref.decode(q, ref.dequantized(fmt, k, ks, 16), ref.dequantized(fmt, v, vs, 16),
                            lambda b, t: t, lens, pos, window, sinks, 0.088)
    ref.check_output(run(cache, q, lens, pos, n, window, sinks, 0.088), want, mass)


def test_decode_rows_at_their_own_positions():
    """Rows need not be the last ones nor in order: some before the window of
    others, some without a position, some past the sequence."""
    cache, q, k, v, lens, _, slot = build(gq.LINEAR, 2, 5, 8, 2, 64, 300, 400, 0, 0, 4, 21)
    pos = torch.tensor([299, 0, -1, 17, 120, 399, 500, -7, 3, 200], dtype=torch.int32)
    want, mass = ref.decode(q, k.double(), v.double(), slot, lens, pos, 40, 4, 0.125)
    got = run(cache, q, lens, pos, 400, 40, 4, 0.125)
    ref.check_output(got, want, mass, weight_bits=16)
    assert not got[0, 2].any() and not got[1, 2].any()


def test_decode_values_that_are_not_finite():
    """A NaN or an infinity reaches the rows that attend its key, no other."""
    cache, q, k, v, lens, pos, slot = build(gq.LINEAR, 1, 4, 4, 2, 128, 200, 200, 0, 50, 4, 5)
    v[199, 0, 3], v[198, 1, 7], v[147, 0, 9] = NAN, float("inf"), NAN
    v[198, 1, 100], v[2, 1, 64] = float("-inf"), NAN
    cache.v.copy_(v)
    got = run(cache, q, lens, pos, 200, 50, 4, 0.1)[0].cpu()   # rows at 196 .. 199
    finite = torch.isfinite(got)
    want = torch.ones_like(finite)
    want[3, :2, 3] = False          # key 199: the last row
    want[2:, 2:, 7] = want[2:, 2:, 100] = False
    want[0, :2, 9] = False          # key 147 is in the window of the row at 196 alone
    want[:, 2:, 64] = False         # a sink: every row
    assert torch.equal(finite, want)
    k[199, 0, 5] = NAN              # a key: its rows whole
    cache.k.copy_(k)
    finite = torch.isfinite(run(cache, q, lens, pos, 200, 50, 4, 0.1)[0].cpu())
    want[3, :2] = False
    assert torch.equal(finite, want)


@pytest.mark.parametrize("D,R,B,hi,window", [
    (128, 1, 1, 900, 0), (64, 1, 1, 900, 0), (128, 5, 2, 2000, 1800), (64, 5, 2, 2000, 0),
    (128, 1, 1, 40000, 0), (64, 2, 60, 700, 500)])
def test_decode_infinite_values(D, R, B, hi, window):
    """An infinity in V makes the element of every row that attends its key infinite,
    with its sign, however small the key's weight is, infinities of both signs a NaN;
    the other elements are as without it."""
    Hq, H = 8, 2
    cache, q, k, v, lens, pos, slot = build(gq.LINEAR, B, R, Hq, H, D, hi, hi, 0, window, 4, D + R)
    inf = float("inf")
    for b in range(B):
        base = b * hi
        for key, h, d, x in ((0, 0, 3, inf), (2, 1, 5, -inf), (hi - 1, 0, 9, inf),
                             (hi - 300, 1, 0, inf), (hi - 301, 1, D - 1, -inf),
                             (hi - 400, 0, 20, inf), (hi - 17, 0, 20, -inf),
                             (hi - 250, 0, 31, inf)):
            v[base + key, h, d] = x
        # a weight of some 2^-200 of the largest
        k[base + hi - 250, 0] = -13 * q[b, 0, 0]
    cache.k.copy_(k)
    cache.v.copy_(v)
    want, _ = ref.decode(q, k.double(), v.double(), slot, lens, pos, window, 4, D ** -0.5)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run(cache, q, lens, pos, hi, window, 4, D ** -0.5, err).cpu()
    assert int(err) == 0
    plain = torch.isfinite(want)
    assert want[:, 0, 0, 31].eq(inf).all() and want[:, R - 1, 0, 20].isnan().all()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.double()[~plain].nan_to_num(0.0, inf, -inf),
                       want[~plain].nan_to_num(0.0, inf, -inf))
    v[~torch.isfinite(v)] = 0
    want, mass = ref.decode(q, k.double(), v.double(), slot, lens, pos, window, 4, D ** -0.5)
    ref.check_output(got.masked_fill(~plain, 0), want.masked_fill(~plain, 0), mass, weight_bits=16)


def test_calls_on_a_stream_of_their_own():
    """Output and workspace that a call makes belong to the stream it is given,
    as a Stream or a handle; two calls on two streams do not disturb each other."""
    cache, q, k, v, lens, pos, slot = build(gq.LINEAR, 2, 1, 8, 2, 128, 3000, 4000, 0, 0, 0, 7)
    q, lens, pos = q.to(DEV), lens.to(DEV), pos.to(DEV)
    want = gq.attn_decode_sinks(q, cache, lens, pos, 4000, 0, 0, 0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(12):
        s = streams[i % 2]
        outs.append(gq.attn_decode_sinks(q, cache, lens, pos, 4000, 0, 0, 0.1,
                                         stream=s if i % 3 else s.cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    pq = torch.randn(1, 300, 4, 64, device=DEV).bfloat16()
    one = gq.attn_prefill_sinks(pq, pq, pq, 50, 4, 0.1)
    torch.cuda.synchronize()
    two = gq.attn_prefill_sinks(pq, pq, pq, 50, 4, 0.1, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(one, two)


def test_strided_and_misplaced_tensors_are_refused():
    cache, q, k, v, lens, pos, slot = build(gq.LINEAR, 2, 2, 4, 2, 64, 50, 60, 0, 9, 2, 7)
    q, lens, pos = q.to(DEV), lens.to(DEV), pos.to(DEV)
    bad = [(q.transpose(2, 3).contiguous().transpose(2, 3), lens, pos), (q.float(), lens, pos),
           (q, lens.long(), pos), (q, lens, pos[::2]), (q, lens.cpu(), pos), (q, lens[:1], pos)]
    for args in bad:
        with pytest.raises(gq.AttnError):
            gq.attn_decode_sinks(args[0], cache, args[1], args[2], 60, 9, 2, 0.1)
    with pytest.raises(gq.AttnError):
        gq.attn_prefill_sinks(q, q, q[:, ::2], 9, 2, 0.1)


@pytest.mark.parametrize("D,R,per", [(128, 1, 16), (64, 1, 16), (64, 5, 32), (128, 2, 24)])
def test_decode_long_shares(D, R, per):
    """64 requests that name the same pages, hundreds of chunks a share, one to compare with."""
    B, H, Hq, L, window, sinks = 64, 8, 16, 4003, 3500, 70
    cache, q, k, v, lens, pos, slot = build(gq.PAGED, 1, R, Hq, H, D, L, L, per, window, sinks, D + R)
    want, mass = ref.decode(q, k.double(), v.double(), slot, lens, pos, window, sinks, D ** -0.5)
    cache.block_table = cache.block_table.repeat(B, 1).contiguous()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = run(cache, q.repeat(B, 1, 1, 1), lens.repeat(B), pos.repeat(B), L, window, sinks,
              D ** -0.5, err)
    assert int(err) == 0
    ref.check_output(got, want.expand(B, -1, -1, -1), mass.expand(B, -1, -1, -1), weight_bits=16)


def test_decode_past_the_tables_of_one_launch():
    """More requests than one launch's tables hold, most of them short."""
    g = gen(1)
    B, H, D, per = 600, 1, 64, 40
    lens = torch.randint(0, per + 1, (B,), generator=g, dtype=torch.int32)
    k, v = (torch.randn(B * per, H, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(B, 1, 2, D, generator=g).bfloat16()
    pos = lens - 1
    want, mass = ref.decode(q, k.double(), v.double(), lambda b, t: b * per + t, lens, pos, 9, 2,
                            0.2)
    cache = gq.KVCache(gq.LINEAR, k.to(DEV), v.to(DEV), slots_per_seq=per)
    ref.check_output(run(cache, q, lens, pos, per, 9, 2, 0.2), want, mass, weight_bits=16)


def test_decode_offsets_past_32_bits():
    """A cache of more than 2^32 bytes a tensor, its last request at the end."""
    per, H, D = 1 << 23, 4, 128
    k, v = (torch.zeros(per, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    g = gen(3)
    n, window, sinks = per, 48, 4
    at = torch.cat([torch.arange(sinks), torch.arange(n - window, n)])
    small = [torch.randn(len(at), H, D, generator=g).bfloat16() for _ in range(2)]
    k[at.to(DEV)], v[at.to(DEV)] = small[0].to(DEV), small[1].to(DEV)
    q = torch.randn(1, 1, 8, D, generator=g).bfloat16()
    lens, pos = torch.tensor([n], dtype=torch.int32), torch.tensor([n - 1], dtype=torch.int32)
    cache = gq.KVCache(gq.LINEAR, k, v, slots_per_seq=per)
    got = run(cache, q, lens, pos, n, window, sinks, 0.1)
    m = torch.tensor([len(at)], dtype=torch.int32)
    want, mass = ref.decode(q, small[0].double(), small[1].double(), lambda b, t: t, m, m - 1, 0,
                            0, 0.1)
    ref.check_output(got, want, mass, weight_bits=16)


@pytest.mark.parametrize("B,T,Hq,H,D,window,sinks", [
    (1, 1, 2, 1, 64, 4, 2),
    (2, 130, 4, 2, 128, 16, 3),
    (1, 515, 4, 4, 64, 1, 1),
    (1, 700, 6, 2, 128, 200, 129),      # sinks past one tile
    (2, 900, 2, 1, 64, 130, 4),
    (1, 640, 4, 2, 128, 64, 1000),      # more sinks than tokens
    (1, 400, 4, 2, 64, 1000, 4),        # a window past the sequence
    (1, 300, 4, 2, 64, 0, 4),           # no window
    (1, 2100, 40, 8, 128, 333, 250),    # two query tiles a CTA
])
def test_prefill(B, T, Hq, H, D, window, sinks):
    g = gen(T + D)
    q = torch.randn(B, T, Hq, D, generator=g).bfloat16()
    k, v = (torch.randn(B, T, H, D, generator=g).bfloat16() for _ in range(2))
    rows = slice(None)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = gq.attn_prefill_sinks(q.to(DEV), k.to(DEV), v.to(DEV), window, sinks, D ** -0.5,
                                err=err)
    assert int(err) == 0
    heads = slice(0, min(Hq, 8 * (Hq // H)), max(1, Hq // 8))
    kv = [h // (Hq // H) for h in range(*heads.indices(Hq))]
    want, mass = ref.prefill(q[:, rows, heads], k[:, :, kv], v[:, :, kv], window, sinks, D ** -0.5)
    ref.check_output(got[:, rows, heads], want, mass)


@pytest.mark.parametrize("sinks", [15, 16, 17, 32, 33, 129, 150, 160, 161])
@pytest.mark.parametrize("group", [1, 5])
def test_prefill_tiles_of_sinks(sinks, group):
    """head_dim 64: a last tile of 1 to 32 sinks or more, behind a whole tile or none,
    walked at different places by the heads of a group; a NaN in V behind the sinks is
    reported and taken as 0."""
    g = gen(sinks + group)
    T, H, D, window = 800, 2, 64, 90
    q = torch.randn(1, T, H * group, D, generator=g).bfloat16()
    k, v = (torch.randn(1, T, H, D, generator=g).bfloat16() for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for behind in (None, 0, 1, 5):
        if behind is not None:
            v[0, sinks + behind, 1, 7 * behind] = NAN
        err.zero_()
        got = gq.attn_prefill_sinks(q.to(DEV), k.to(DEV), v.to(DEV), window, sinks, D ** -0.5,
                                    err=err)
        assert int(err) == (0 if behind is None else gq.ATTN_ERR_UNSUPPORTED)
        want, mass = ref.prefill(q, k, v.nan_to_num(0.0), window, sinks, D ** -0.5)
        ref.check_output(got, want, mass)


def test_prefill_values_that_are_not_finite():
    """K and V behind a row do not reach it; a NaN in V is reported."""
    g = gen(2)
    q = torch.randn(1, 300, 4, 64, generator=g).bfloat16()
    k, v = (torch.randn(1, 300, 2, 64, generator=g).bfloat16() for _ in range(2))
    clean = gq.attn_prefill_sinks(q.to(DEV), k.to(DEV), v.to(DEV), 32, 4, 0.1)
    k[0, 290:], v[0, 290:] = NAN, NAN
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = gq.attn_prefill_sinks(q.to(DEV), k.to(DEV), v.to(DEV), 32, 4, 0.1, err=err)
    assert int(err) == gq.ATTN_ERR_UNSUPPORTED
    assert torch.equal(got[:, :290], clean[:, :290])


@pytest.mark.parametrize("D,group,sinks,window,T", [
    (64, 1, 1, 150, 600),     # the tile of few sinks
    (64, 7, 20, 200, 500),    # ... of 17 to 32, and heads that start at other tiles
    (64, 2, 60, 150, 400),    # a whole tile of sinks
    (128, 1, 1, 150, 600),
    (128, 4, 130, 128, 700),  # two tiles of sinks
])
def test_prefill_small_weights_beside_a_sink(D, group, sinks, window, T):
    """A sink with values of zero takes most of a row.  Key j of the window has
    2^(-j / 2) of its weight and a value that stands alone in dim j: each weight
    shows by itself, and down to 2^-20 of the sink's keeps the precision of one
    rounding to 11 bits."""
    n = 41
    q, k, v = (torch.zeros(1, T, h, D) for h in (group, 1, 1))
    q[..., 0] = 1.0
    k[..., 0] = -60.0
    k[0, sinks - 1, 0, 0] = 0.0
    for j in range(n):
        k[0, T - n - 5 + j, 0, 0] = -j / 2
        v[0, T - n - 5 + j, 0, j] = 96.0
    q, k, v = (x.bfloat16() for x in (q, k, v))
    scale = math.log(2.0)
    got = gq.attn_prefill_sinks(q.to(DEV), k.to(DEV), v.to(DEV), window, sinks, scale)
    want, mass = ref.prefill(q, k, v, window, sinks, scale)
    ref.check_output(got, want, mass)


def test_prefill_agrees_with_decode():
    """The last rows of a prompt, prefilled and decoded from a paged cache."""
    g = gen(4)
    T, Hq, H, D, window, sinks, bs = 450, 8, 2, 128, 100, 5, 16
    q = torch.randn(1, T, Hq, D, generator=g).bfloat16().to(DEV)
    k, v = (torch.randn(1, T, H, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    whole = gq.attn_prefill_sinks(q, k, v, window, sinks, 0.09)
    pages = -(-T // bs)
    table = torch.randperm(pages, generator=g).int().view(1, -1).to(DEV)
    kc, vc = (torch.zeros(pages * bs, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = gq.KVCache(gq.PAGED, kc, vc, block_table=table, block_size=bs)
    t = torch.arange(T, device=DEV)
    gq.attn_kv_append(k[0], v[0], table[0, t // bs].long() * bs + t % bs, cache)
    lens = torch.tensor([T], dtype=torch.int32, device=DEV)
    pos = torch.arange(T - 3, T, dtype=torch.int32, device=DEV)
    last = gq.attn_decode_sinks(q[:, -3:].contiguous(), cache, lens, pos, T, window, sinks, 0.09)
    want, mass = ref.prefill(q.cpu(), k.cpu(), v.cpu(), window, sinks, 0.09)
    ref.check_output(whole, want, mass)
    ref.check_output(last, want[:, -3:], mass[:, -3:], weight_bits=16)
