"""Shared prefixes where their parts meet odd bounds: shares of own keys that hold none,
small values, scales at their ends, positions and lengths near the ends of int32."""
import pytest
import torch

import gqa_attention_kv_gb300 as gq
import kv_reference as ref
from test_gpu_shared import DEV, DTYPE, Case, one_group

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,n,H,D", [("bf16", 60, 1, 128), ("bf16", 200, 4, 64),
                                       ("int8", 120, 2, 64), ("e4m3", 37, 8, 128)])
def test_shares_that_lie_in_gaps(fmt, n, H, D):
    """Own keys of 1 to 20: a share of four chunks of 34 a unit holds keys in one of eight, and
    the others follow one another without work between them."""
    c = Case(fmt, gq.LINEAR, one_group(n, 48), [1 + (7 * i) % 20 for i in range(n)], 1, 2 * H, H, D,
             16, n + D)
    want = c.check()
    need = gq.attn_decode_shared_workspace_size(c.cache, n, 1, 2 * H, c.longest, c.max_prefix)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for _ in range(50):
        assert torch.equal(c.run(workspace=ws), want)


def weights(c, b, r, h, scale):
    """Softmax weights of the keys that a row attends (a head of KV head h's group), and their
    slots."""
    n, pos = int(c.lens[b]), int(c.pos[b * c.R + r])
    slots = torch.tensor([c.slot(b, t) for t in range(min(n, pos + 1))
                          if not c.window or pos - t < c.window])
    G = c.q.shape[2] // c.H
    s = scale * (c.q[b, r, h * G:(h + 1) * G].double() @ c.kd[slots, h].T)
    return torch.softmax(s, -1), slots


def check_spread(c):
    """A softmax over n spread keys is about sqrt(n) smaller than the sum of |p v|, so a bound by
    that sum does not see what an output's own magnitude loses.  Bounds: the output's rounding,
    2^-8 of it; 2^-13 of sum |p v| for scores and sums in 32 bits; weights, each off by at most
    2^-11 of itself by itself, by Hoeffding within 7 2^-11 sqrt(sum p^2 v^2) but for one in 10^10;
    and the parts' outputs, whose rounding is 2^-11 of sums of p v over the part, of the same
    size again (values of either sign)."""
    scale = c.D ** -0.5
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = c.run(err=err).double().cpu()
    assert int(err) == 0
    want, mass = c.want()
    G = c.q.shape[2] // c.H
    for b in range(c.q.shape[0]):
        for r in range(c.R):
            for h in range(c.H):
                p, slots = weights(c, b, r, h, scale)
                size = (p ** 2 @ c.vd[slots, h] ** 2).sqrt()
                at = (b, r, slice(h * G, (h + 1) * G))
                bound = 2.0 ** -8 * want[at].abs() + 2.0 ** -13 * mass[at] + 14 * 2.0 ** -11 * size
                over = ((got[at] - want[at]).abs() / bound).max().item()
                assert over <= 1.0, f"{over:.3f} of the bound"


def put_values(c, v):
    """Values [slots, H, D] (64 bits) of a case; its cache holds them rounded."""
    if c.fmt == "bf16":
        v = v.float().bfloat16()
        c.vd, raw = v.double(), v
    else:
        raw = ref.encode("e4m3", v, torch.tensor(1.0, dtype=torch.float64))
        c.vd = ref.code_values("e4m3", raw)
    c.cache.v.copy_(raw.to(DEV))


@pytest.mark.parametrize("low", [0, 10, 14, 16, 20, 24, 40, 60, 75])
@pytest.mark.parametrize("n,D,own", [(2, 128, 3), (40, 64, 1)])
def test_small_values(low, n, D, own):
    """bf16 values of 2^-low over 4,096 shared keys keep what attn_decode keeps of them: lone
    tiles and pairs."""
    c = Case("bf16", gq.LINEAR, one_group(n, 4096 if n == 2 else 1500), [own] * n, 1, 8, 2, D, 16,
             low + n, hole=False)
    put_values(c, c.vd * 2.0 ** -low)
    check_spread(c)
    c.check()


def test_small_codes():
    """E4M3 codes of a few steps of its smallest, over 4,096 keys."""
    c = Case("fp8", gq.LINEAR, one_group(2, 4096), [3, 5], 1, 8, 2, 128, 16, 2, hole=False)
    put_values(c, torch.randn(c.vd.shape, generator=torch.Generator().manual_seed(3),
                              dtype=torch.float64) * 2.0 ** -8)
    check_spread(c)


def test_the_counter_of_shares_is_left_at_zero():
    """... by calls of one launch and of two, whatever lies behind the workspace's counters; a
    decode and a window with sinks find their counters as they need them."""
    few = Case("bf16", gq.LINEAR, one_group(5, 300), [7, 8, 40, 1, 90], 1, 8, 2, 128, 16, 1, hole=False)
    many = Case("bf16", gq.LINEAR, one_group(300, 40), [1 + i % 50 for i in range(300)], 1, 2, 1, 64,
                8, 2, hole=False)
    flat = Case("bf16", gq.LINEAR, [(0, 0), (1, 0)], [900, 100], 1, 8, 2, 128, 16, 3, hole=False)
    need = max(gq.attn_decode_shared_workspace_size(c.cache, c.q.shape[0], 1, c.q.shape[2], c.longest,
                                                    c.max_prefix) for c in (few, many))
    need = max(need, gq.attn_decode_workspace_size(flat.cache, 2, 1, 8, 900))
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    wants = few.check(), many.check()
    a = [x.to(DEV) for x in (flat.lens, flat.pos)]
    exact, mass = flat.want()
    for _ in range(3):
        for c, want in zip((few, many), wants):
            assert torch.equal(c.run(workspace=ws), want)
            assert not ws[:1024].any()
        ref.check_output(gq.attn_decode(flat.q.to(DEV), flat.cache, *a, 900, 0, 128 ** -0.5,
                                        workspace=ws), exact, mass)
        ws[-8192:] = 0xFF  # (partial states)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("large,small", [(2.0 ** 10, 2.0 ** -20), (1.0, 2.0 ** -45),
                                         (2.0 ** 12, 0.0), (0.0, 2.0 ** -30)])
def test_values_of_different_size_along_the_prefix(n, large, small):
    """Key tiles of large values, of small ones and of zeros; rows that attend all of them, the
    first ones only, or by their window the last ones only, within the bound of what they attend."""
    c = Case("bf16", gq.LINEAR, one_group(n, 900), [40] * n, 1, 8, 2, 128, 16, 5, hole=False)
    size = torch.ones(c.vd.shape[0], 1, 1, dtype=torch.float64) * small
    size[:256] = large
    size[640:] = small * 2.0 ** -7
    put_values(c, c.vd * size)
    c.lens = torch.tensor([[940, 200, 700][i % 3] for i in range(n)], dtype=torch.int32)
    c.pos = c.lens - 1
    for c.window in (0, 60):
        c.check()
    # weights that fall to the first keys by 2^-40, or rise to them
    c.q[:] = 0
    c.q[..., 0] = 1
    c.window = 0
    for ends in ((0.0, 27.0), (27.0, 0.0)):
        c.kd[:, :, 0] = torch.linspace(*ends, c.kd.shape[0])[:, None].bfloat16().double()
        c.cache.k.copy_(c.kd.bfloat16().to(DEV))
        c.check(scale=1.0)


def test_values_that_are_not_finite_beside_small_ones():
    """A NaN is taken as 0 and reported, and the tile's other values keep their bits."""
    c = Case("bf16", gq.PAGED, one_group(5, 700), [3, 4, 5, 6, 7], 1, 8, 2, 128, 16, 5, hole=False)
    put_values(c, c.vd * 2.0 ** -30)
    c.check()
    at = c.slot(0, 150)
    c.cache.v[at, 1, 7] = float("nan")
    c.vd[at, 1, 7] = 0.0
    want, mass = c.want()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = c.run(err=err)
    assert int(err) == gq.ATTN_ERR_UNSUPPORTED
    ref.check_output(got, want, mass, weight_bits=10)


def test_absent_pages_beside_small_values():
    """The second reading of a tile skips a page that is not in the pool too."""
    c = Case("bf16", gq.PAGED, one_group(3, 600), [3, 4, 5], 1, 8, 2, 64, 16, 6, hole=False)
    put_values(c, c.vd * 2.0 ** -30)
    c.cache.block_table[0, 5] = -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = c.run(err=err)
    assert int(err) == gq.ATTN_ERR_BOUNDS
    slot = c.slot
    c.slot = lambda b, t: -1 if 80 <= t < 96 else slot(b, t)
    want, mass = c.want()
    ref.check_output(got, want, mass, weight_bits=10)


@pytest.mark.parametrize("fmt,bs", [("bf16", 1 << 20), ("bf16", 300), ("int8", 320)])
def test_prefixes_that_end_near_2_31(fmt, bs):
    """Under a window, with two pages that serve every table entry: one that is not there is
    reported and masked, though its end lies past 2^31."""
    end, window, D = 2 ** 31 - 270, 700, 64
    base = end - 1000  # (the reference counts from here on)
    g = torch.Generator().manual_seed(bs)
    pool, more = torch.randn(2, 2 * bs, 1, D, generator=g).bfloat16(), {}
    if fmt == "int8":
        pool = (pool * 30).clamp(-127, 127).to(torch.int8)
        scale = torch.full((2 * bs // 16, 1), 2.0 ** -5, device=DEV)
        more = dict(dtype=DTYPE[fmt], k_scale=scale, v_scale=scale.clone(), scale_block=16)
    values = pool.double() if fmt == "bf16" else pool.double() * 2.0 ** -5
    table = torch.zeros(3, -(-(end + 10) // bs), dtype=torch.int32, device=DEV)
    table[:, 1::2] = 1
    cache = gq.KVCache(gq.PAGED, pool[0].to(DEV), pool[1].to(DEV), block_table=table, block_size=bs,
                       **more)
    q = torch.randn(2, 1, 4, D, generator=g).bfloat16()
    i32 = dict(dtype=torch.int32)
    lens = torch.tensor([end + 3, end + 9], **i32)
    args = [x.to(DEV) for x in (lens, lens - 1, torch.full((2,), 2, **i32),
                                torch.full((2,), end, **i32))]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def check(absent):
        def slot(b, t):
            t += base
            return -1 if t < end and t // bs == absent else t // bs % 2 * bs + t % bs

        want, mass = ref.decode(q, values[0], values[1], slot, lens - base,
                                lens - 1 - base, window, 0, D ** -0.5)
        got = gq.attn_decode_shared(q.to(DEV), cache, *args, end + 10, end, window, D ** -0.5,
                                    err=err)
        ref.check_output(got, want, mass, weight_bits=10)

    check(-1)
    assert int(err) == 0
    absent = (end - 300) // bs
    table[2, absent] = -1
    check(absent)
    assert int(err) == gq.ATTN_ERR_BOUNDS


@pytest.mark.parametrize("fmt,D", [("bf16", 64), ("int8", 64), ("e4m3", 128)])
def test_any_number_of_groups(fmt, D):
    """The CTAs at work follow the groups, which a replay of one graph changes: one, a few, as many
    as requests, none, equal lengths in other rows, one row at other lengths."""
    n = 70
    c = Case(fmt, gq.LINEAR, one_group(n, 90), [1 + i % 9 for i in range(n)], 1, 4, 2, D, 16, 9 + D,
             hole=False)
    need = gq.attn_decode_shared_workspace_size(c.cache, n, 1, 4, c.longest, c.max_prefix)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    q, lens, pos, prows, plens = (x.to(DEV) for x in (c.q, c.lens, c.pos, c.prows, c.plens))
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    c.run()
    with torch.cuda.graph(graph):
        gq.attn_decode_shared(q, c.cache, lens, pos, prows, plens, c.longest, c.max_prefix, 0,
                              D ** -0.5, out=out, workspace=ws)
    for i, of in enumerate([lambda b: (0, 90), lambda b: (b // 30, 90), lambda b: (b, 90),
                            lambda b: (0, 90 if b < 35 else 40), lambda b: (b, 0),
                            lambda b: (b // 4, 30 + b // 4), lambda b: (b % 2, 90),
                            lambda b: (0, 90 * (b % 2))]):
        at = [of(b) for b in range(n)]
        c.prows.copy_(torch.tensor([a[0] for a in at]))
        c.plens.copy_(torch.tensor([a[1] for a in at]))
        prows.copy_(c.prows), plens.copy_(c.plens)
        graph.replay()
        want, mass = c.want()
        ref.check_output(out, want, mass, weight_bits=10)


def test_more_groups_than_a_block_counts_at_once():
    """1,300 requests in 700 groups."""
    prefix, first = [], 0
    for i in range(700):
        size = 1 + (i % 7 < 6)
        prefix += [(first, 0 if i % 11 == 5 else 10 + i % 60)] * size
        first += size
    Case("bf16", gq.PAGED, prefix, [1 + i % 4 for i in range(first)], 1, 2, 1, 64, 16, 31).check()


def put_scales(c, ks, vs, sb=16):
    """Scales [slots / sb, heads] of a case (64 bits); smaller ones than 2^-64 are read as that."""
    code = {"k": c.cache.k, "v": c.cache.v}
    for name, x in (("k", ks.float()), ("v", vs.float())):
        getattr(c.cache, name + "_scale").copy_(x.to(DEV))
        values = ref.dequantized(c.fmt, code[name].cpu(), x.clamp(min=ref.FLOOR), sb)
        setattr(c, name + "d", values)


@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("fmt,kind,D", [("e4m3", gq.LINEAR, 128), ("int8", gq.PAGED, 64),
                                        ("int8", gq.LINEAR, 128), ("e4m3", gq.PAGED, 64)])
def test_scales_at_their_ends(fmt, kind, D, n):
    """Values' scales from 0 to 2^119 (codes of 127 and 448 end below bf16's 2^128) and keys' from 0
    on; blocks side by side, across the border of prefix and own keys too, that differ by up to 2^100
    (a weight times vs / vs_max is held times 2^7 in float32, which ends at 2^-126: 2^-33 of a weight
    whose scale is 2^-100 of the largest, 250 of which are nothing beside the bound's 2^-13)."""
    c = Case(fmt, kind, one_group(n, 200), [1 + i % 50 for i in range(n)], 1, 8, 2, D, 16, n + D,
             hole=False)
    shape = c.cache.k_scale.shape
    g = torch.Generator().manual_seed(D + n)
    ones = torch.ones(shape, dtype=torch.float64)
    usual = ones * (1.0 / 128 if fmt == "int8" else 1.0 / 64)

    def powers(lo, hi):
        return 2.0 ** torch.randint(lo, hi + 1, shape, generator=g).double()

    for ks, vs in ((usual, ones * 0.0), (usual, ones * 2.0 ** -70), (usual, ones * 2.0 ** -64),
                   (usual, ones * 2.0 ** 119), (usual, powers(-30, 30)), (usual, powers(-64, 36)),
                   (usual, powers(19, 119)),
                   (ones * 0.0, usual), (ones * 2.0 ** -64, powers(-10, 10)),
                   (usual * powers(-8, 2), usual), (usual * powers(-30, 0), powers(-3, 3))):
        put_scales(c, ks, vs)
        c.check()


@pytest.mark.parametrize("fmt,kind", [("int8", gq.LINEAR), ("e4m3", gq.PAGED), ("fp8", gq.LINEAR)])
def test_positions_at_the_ends_of_int32(fmt, kind):
    c = Case(fmt, kind, one_group(5, 300), [4] * 5, 2, 8, 2, 128, 16, 6, hole=False)
    low, high = -2 ** 31, 2 ** 31 - 1
    c.pos = torch.tensor([low, 303, 302, low + 1, -2, low + 299, 302, high, 300, low],
                         dtype=torch.int32)
    for c.window in (0, 2 ** 31 - 1, 20):
        got = c.check()
        assert not got[0, 0].any() and not got[1, 1].any() and not got[2].any()


@pytest.mark.parametrize("n,per,kind", [(2, 16, gq.LINEAR), (40, 16, gq.PAGED), (3, 5, gq.PAGED)])
def test_values_whose_size_jumps(n, per, kind):
    """Key tiles each of a size that the one before does not foretell, the first one's later keys
    too; pages that are gathered row by row."""
    c = Case("bf16", kind, one_group(n, 1500), [1 + i % 30 for i in range(n)], 1, 8, 2, 128, per, n,
             hole=False)
    lead = torch.tensor([c.slot(0, t) for t in range(1500)])
    g = torch.Generator().manual_seed(n)
    for first in (0, -40, 12):
        size = torch.ones(c.vd.shape[0], 1, 1, dtype=torch.float64) * 2.0 ** -10
        powers = torch.randint(-60, 13, (12,), generator=g)
        powers[0] = first
        size[lead, 0, 0] = 2.0 ** powers[torch.arange(1500) // 128].double()
        size[lead[100:128]] *= 2.0 ** (-20 if first > 0 else 10)
        values = torch.randn(c.vd.shape, generator=g, dtype=torch.float64)
        put_values(c, (values * size).clamp(-60000, 60000))
        c.check()
        # rows that only attend one tile's keys, by their windows
        c.lens = torch.tensor([130 + 37 * (i % 30) for i in range(n)], dtype=torch.int32)
        c.pos, c.window = c.lens - 1, 60
        c.check()
        c.lens = c.plens + torch.tensor([1 + i % 30 for i in range(n)], dtype=torch.int32)
        c.pos, c.window = c.lens - 1, 0


@pytest.mark.parametrize("n,groups,H,prefix,own", [(7, 3, 8, 300, 40), (120, 64, 1, 900, 3),
                                                   (60, 31, 2, 200, 2), (90, 45, 4, 40, 1)])
def test_more_pieces_than_ctas_at_work(n, groups, H, prefix, own):
    """Groups between the powers of two that CTAs are counted for: pieces past their number are taken
    in a second round, by the CTAs at work only."""
    at = [(i * groups // n) for i in range(n)]
    lead = [at.index(a) for a in at]
    Case("bf16", gq.LINEAR, [(b, prefix + a % 7) for b, a in zip(lead, at)],
         [1 + i % own for i in range(n)], 1, 2 * H, H, 64, 16, n + groups).check()
