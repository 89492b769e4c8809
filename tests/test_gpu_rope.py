"""Norms of queries and keys with their rotary embedding, alone and written to a
cache by the same launch."""
import math

import pytest
import torch

import gqa_attention_kv_gb300 as gq

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF, PAIRS = gq.ATTN_ROPE_HALF, gq.ATTN_ROPE_PAIRS


def gen(seed):
    return torch.Generator().manual_seed(seed)


def turned(x, pos, inv, layout, factor, weight, eps):
    """The definition in 64 bits: rows x [n, heads, D].  Returns the result and, per
    element, the magnitude that roundings act on."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    y, size = x.clone(), x.abs()
    half = inv.numel()
    a = pos.double()[:, None, None] * inv.double()
    c, s = factor * a.cos(), factor * a.sin()
    i = torch.arange(half)
    one, two = (i, i + half) if layout == HALF else (2 * i, 2 * i + 1)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    both = (x[..., one].abs() + x[..., two].abs()) * abs(factor)
    size[..., one] = size[..., two] = both
    return y, size


# One rounding to bf16 (half a step, 2^-8 of the value), and float32 before it: an angle is
# within 2^-31 of a turn and, as a float of half turns, 2^-25 half turns of its value
# (1.1e-7 radians in all); sincospif, two products and a sum are within 5 half steps of
# 2^-24 and its 2 steps (4e-7 in all); a norm adds its sum's error (a tree of 8 and 4
# additions: 2^-21 / 2), 2 steps of rsqrtf, two products (7e-7).  Under 2^-19 in all.
def check(got, want):
    y, size = want
    got = got.double().cpu()
    bound = 2.0 ** -8 * y.abs() + 2.0 ** -19 * size + 1e-38
    over = ((got - y).abs() / bound).max().item()
    assert over <= 1.0, f"{over:.3f} of the bound"


def make(n, Hq, H, D, rot, layout, norm, seed, far=1000, factor=1.0, strided=True):
    g = gen(seed)
    fused = torch.randn(n, Hq + 2 * H, D, generator=g).bfloat16()
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]
    pos = torch.randint(0, far, (n,), generator=g).int()
    inv, _ = gq.rope_frequencies(rot)
    weights = [1 + 0.3 * torch.randn(D, generator=g) for _ in range(2)] if norm else [None, None]
    rope = gq.Rope(inv.to(DEV) if rot else None, layout, factor,
                   *(w if w is None else w.to(DEV) for w in weights), eps=1e-5)
    dev = fused.to(DEV)
    dq, dk, dv = dev[:, :Hq], dev[:, Hq:Hq + H], dev[:, Hq + H:]
    if not strided:
        dq, dk, dv = (x.contiguous() for x in (dq, dk, dv))
    want = [turned(x, pos, inv, layout, factor, w, 1e-5) for x, w in zip((q, k), weights)]
    return (dq, dk, dv, pos.to(DEV), rope), want, v


@pytest.mark.parametrize("layout", [HALF, PAIRS])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("n,Hq,H,D,rot", [
    (1, 1, 1, 64, 64), (1, 28, 4, 128, 128), (3, 7, 1, 128, 64), (65, 32, 8, 128, 32),
    (130, 5, 3, 64, 16), (33, 12, 2, 64, 48), (17, 8, 8, 128, 96), (9, 4, 2, 128, 20),
    (9, 3, 3, 64, 2), (4, 4, 1, 128, 126), (2500, 28, 4, 128, 128), (5, 3, 2, 64, 0)])
def test_rope(layout, norm, n, Hq, H, D, rot):
    (q, k, _, pos, rope), want, _ = make(n, Hq, H, D, rot, layout, norm, n + rot + D)
    for got, w in zip(gq.attn_qk_rope(q, k, pos, rope), want):
        check(got, w)


@pytest.mark.parametrize("layout", [HALF, PAIRS])
def test_far_positions(layout):
    """Up to the largest int32 and below zero; frequencies of every size and sign."""
    n, D = 200, 128
    (q, k, _, _, _), _, _ = make(n, 4, 2, D, D, layout, False, 5)
    pos = torch.cat([torch.tensor([0, 1, 2 ** 31 - 1, -1, -2 ** 31, 2 ** 24 + 1]),
                     torch.randint(10 ** 5, 2 ** 31 - 1, (n - 6,), generator=gen(6))]).int()
    inv = torch.rand(D // 2, generator=gen(7)) * 2.0 ** torch.randint(-40, 5, (D // 2,),
                                                                      generator=gen(8))
    inv[:6] = torch.tensor([0.0, 1.0, -1.0, 2.0 ** -149, 3.0e-39, 1.0e-30])
    rope = gq.Rope(inv.float().to(DEV), layout, 1.25)
    a = pos.double()[:, None] * inv.float().double()  # 55 bits: reduced exactly below
    got = gq.attn_qk_rope(q, k, pos.to(DEV), rope)
    # p * inv of up to 2^36 radians in 64 bits is off by 2^-17: reduce with integers instead
    from fractions import Fraction
    turn = Fraction(884279719003555, 281474976710656)  # pi to 2^-50 ... refined:
    two_pi = Fraction(int("6283185307179586476925286766559005768394338798750211641949889184615632"),
                      10 ** 69)
    assert abs(two_pi - 2 * turn) < Fraction(1, 2 ** 40)
    exact = torch.empty_like(a)
    for i, p in enumerate(pos.tolist()):
        for j, f in enumerate(inv.float().tolist()):
            x = Fraction(f) * p
            exact[i, j] = float(x - two_pi * (x // two_pi))
    for x, y in zip((q, k), got):
        x = x.double().cpu()
        c, s = 1.25 * exact.cos()[:, None], 1.25 * exact.sin()[:, None]
        one, two = (slice(0, D // 2), slice(D // 2, D)) if layout == HALF else \
            (slice(0, D, 2), slice(1, D, 2))
        want, size = torch.empty_like(x), torch.empty_like(x)
        want[..., one] = x[..., one] * c - x[..., two] * s
        want[..., two] = x[..., two] * c + x[..., one] * s
        size[..., one] = size[..., two] = 1.25 * (x[..., one].abs() + x[..., two].abs())
        # the fraction of a turn: frequencies below 2^5 to 2^-26 of a turn, within what the
        # float of half turns is allowed
        check(y, (want, size))


def test_in_place_and_one_sided_norms():
    (q, k, _, pos, rope), want, _ = make(70, 6, 2, 128, 128, HALF, True, 3, strided=False)
    first = gq.attn_qk_rope(q, k, pos, rope)
    a, b = q.clone(), k.clone()
    got = gq.attn_qk_rope(a, b, pos, rope, q_out=a, k_out=b)
    assert got[0] is a and torch.equal(a, first[0]) and torch.equal(b, first[1])
    bare = gq.attn_qk_rope(q, k, pos, gq.Rope(rope.inv_freq, HALF))
    mixed = gq.attn_qk_rope(q, k, pos, gq.Rope(rope.inv_freq, HALF, k_weight=rope.k_weight,
                                               eps=1e-5))
    assert torch.equal(mixed[0], bare[0]) and torch.equal(mixed[1], first[1])
    mixed = gq.attn_qk_rope(q, k, pos, gq.Rope(rope.inv_freq, HALF, q_weight=rope.q_weight,
                                               eps=1e-5))
    assert torch.equal(mixed[0], first[0]) and torch.equal(mixed[1], bare[1])


@pytest.mark.parametrize("D", [64, 128])
def test_large_small_and_odd_values(D):
    """Squares past float32, rows of zeros, and what is not finite: it stays in its row
    (norm) or pair (rotation)."""
    g = gen(4)
    x = torch.randn(6, 2, D, generator=g)
    x[1] *= 1e30
    x[2] = 0
    x[3] *= 1e-30
    x[4, 0, 3] = math.inf
    x[4, 1, D // 2] = math.nan
    x = x.bfloat16()
    pos, w = torch.arange(6).int(), torch.rand(D, generator=g) + 0.5
    inv, _ = gq.rope_frequencies(D)
    for weight in (w, None):
        rope = gq.Rope(inv.to(DEV), HALF, 1.0, q_weight=None if weight is None else w.to(DEV),
                       eps=1e-6)
        got = gq.attn_qk_rope(x.to(DEV), x.to(DEV), pos.to(DEV), rope)[0].cpu()
        y, size = turned(x, pos, inv, HALF, 1.0, weight, 1e-6)
        keep = [0, 1, 2, 3, 5]
        check(got[keep], (y[keep], size[keep]))
        if weight is None:
            odd = ~torch.isfinite(got[4])
            assert odd[0].nonzero().flatten().tolist() == [3, 3 + D // 2]
            assert odd[1].nonzero().flatten().tolist() == [0, D // 2]
        else:
            assert torch.isnan(got[4, 1]).all() and torch.isnan(got[4, 0, 3])


def make_cache(kind, dtype, slots, H, D, per, head_major):
    raw = torch.bfloat16 if dtype == gq.ATTN_KV_BF16 else \
        torch.int8 if dtype == gq.ATTN_KV_INT8_SCALED else torch.uint8
    shape = (slots // per, H, per, D) if head_major else (slots, H, D)
    k, v = (torch.zeros(shape, dtype=raw, device=DEV) for _ in range(2))
    more = {}
    if dtype in (gq.ATTN_KV_FP8_E4M3_SCALED, gq.ATTN_KV_INT8_SCALED):
        more = {n: torch.zeros(slots // 16, H, device=DEV) for n in ("k_scale", "v_scale")}
        more["scale_block"] = 16
    if dtype != gq.ATTN_KV_BF16:
        more["k_ref"] = torch.randn(H, D, generator=gen(1)).to(DEV)
    table = torch.arange(slots // per, device=DEV, dtype=torch.int32)[None, :].contiguous()
    return gq.KVCache(kind, k, v, slots_per_seq=per if kind != gq.PAGED else 0,
                      block_table=table if kind == gq.PAGED else None,
                      block_size=per if kind == gq.PAGED else 0, dtype=dtype,
                      layout=gq.ATTN_LAYOUT_BHSD if head_major else gq.ATTN_LAYOUT_BSHD, **more)


@pytest.mark.parametrize("dtype,D,kind,head_major", [
    (dtype, D, kind, head_major)
    for dtype, D in ((gq.ATTN_KV_BF16, 64), (gq.ATTN_KV_BF16, 128), (gq.ATTN_KV_FP8_E4M3, 128),
                     (gq.ATTN_KV_FP8_E4M3_SCALED, 64), (gq.ATTN_KV_INT8_SCALED, 128))
    for kind, head_major in ((gq.LINEAR, False), (gq.PAGED, True), (gq.RING, False))
    # rings of scaled blocks are refused
    if kind != gq.RING or dtype in (gq.ATTN_KV_BF16, gq.ATTN_KV_FP8_E4M3)])
@pytest.mark.parametrize("layout,rot,norm,n", [(HALF, 64, True, 40), (PAIRS, 32, False, 7),
                                               (HALF, 20, True, 1000)])
def test_append_is_rope_then_append(dtype, D, kind, head_major, layout, rot, norm, n):
    """Bit for bit the two calls, for every cache; slots outside are skipped."""
    scaled = dtype in (gq.ATTN_KV_FP8_E4M3_SCALED, gq.ATTN_KV_INT8_SCALED)
    H, per = 3, 32
    (q, k, v, pos, rope), want, v_cpu = make(n, 9, H, D, rot, layout, norm, n)
    slots = (n + 40 + per - 1) // per * per
    at = torch.arange(n) + 5
    if not scaled:
        at = at[torch.randperm(n, generator=gen(2))]
    if n > 3:
        at[2] = slots + 3
    at = at.to(DEV)
    mine = make_cache(kind, dtype, slots, H, D, per, head_major)
    two = make_cache(kind, dtype, slots, H, D, per, head_major)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k_out = torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV)
    qo = gq.attn_qk_rope_append(q, k, v, pos, at, mine, rope, k_out=k_out, err=err)
    assert int(err) == (gq.ATTN_ERR_BOUNDS if n > 3 else 0)
    q2, k2 = gq.attn_qk_rope(q, k, pos, rope)
    gq.attn_kv_append(k2, v.contiguous(), at, two)
    assert torch.equal(qo, q2) and torch.equal(k_out, k2)
    check(qo, want[0])
    for name in ("k", "v") + (("k_scale", "v_scale") if scaled else ()):
        assert torch.equal(getattr(mine, name), getattr(two, name)), name
    # without the extra copy of the keys
    three = make_cache(kind, dtype, slots, H, D, per, head_major)
    gq.attn_qk_rope_append(q, k, v, pos, at, three, rope)
    assert torch.equal(three.k, two.k) and torch.equal(three.v, two.v)


def test_agrees_with_the_rotation_of_decode_append():
    """attn_decode_append's rotary embedding (float32 angles) at near positions."""
    g = gen(9)
    B, Hq, H, D, L = 3, 8, 2, 128, 60
    q, k, v = (torch.randn(B, h, D, generator=g).bfloat16().to(DEV) for h in (Hq, H, H))
    inv = gq.rope_frequencies(D)[0].to(DEV)
    lens = torch.tensor([20, 41, 60], dtype=torch.int32, device=DEV)
    pos, at = lens - 1, (torch.arange(B, device=DEV) * L + lens - 1).long()
    kc, vc = (torch.randn(B * L, H, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    one = gq.KVCache(gq.LINEAR, kc.clone(), vc.clone(), slots_per_seq=L)
    two = gq.KVCache(gq.LINEAR, kc.clone(), vc.clone(), slots_per_seq=L)
    a = gq.attn_decode_append(q[:, None].contiguous(), k, v, at, one, lens, pos, L, 0, 0.09,
                              rope_inv_freq=inv)
    qo = gq.attn_qk_rope_append(q, k, v, pos, at, two, gq.Rope(inv, PAIRS))
    b = gq.attn_decode(qo[:, None].contiguous(), two, lens, pos, L, 0, 0.09)
    assert torch.equal(one.v, two.v)
    # rotated keys: float32 angles of up to 60 radians are off by 2^-19, which may carry an
    # element over a rounding border: a bf16 step, 2^-7 of it, at most
    assert ((one.k.double() - two.k.double()).abs() <= 2.0 ** -7 * two.k.double().abs() + 1e-4).all()
    assert (a.double() - b.double()).abs().max() < 0.05


def test_stream_and_graph():
    (q, k, v, pos, rope), _, _ = make(100, 8, 2, 128, 128, HALF, True, 12)
    plain = gq.attn_qk_rope(q, k, pos, rope)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = gq.attn_qk_rope(q, k, pos, rope, stream=s)
    s.synchronize()
    assert torch.equal(plain[0], on_s[0]) and torch.equal(plain[1], on_s[1])
    cache = make_cache(gq.LINEAR, gq.ATTN_KV_BF16, 128, 2, 128, 128, False)
    at, qo = torch.arange(100, device=DEV), torch.empty_like(plain[0])
    gq.attn_qk_rope_append(q, k, v, pos, at, cache, rope, q_out=qo)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq.attn_qk_rope_append(q, k, v, pos, at, cache, rope, q_out=qo)
    # positions and slots are read by the replay
    pos.add_(17), at.add_(20)
    cache.k.zero_()
    graph.replay()
    want = gq.attn_qk_rope(q, k, pos, rope)
    assert torch.equal(qo, want[0]) and torch.equal(cache.k[20:120], want[1])
    assert not cache.k[:20].any() and torch.equal(cache.v[20:120], v)


def test_refusals_of_tensors():
    (q, k, v, pos, rope), _, _ = make(8, 4, 2, 128, 128, HALF, True, 1)
    cache = make_cache(gq.LINEAR, gq.ATTN_KV_BF16, 32, 2, 128, 32, False)
    at = torch.arange(8, device=DEV)

    def no(call, *a, **kw):
        with pytest.raises(gq.AttnError):
            call(*a, **kw)

    no(gq.attn_qk_rope, q.float(), k, pos, rope)
    no(gq.attn_qk_rope, q.cpu(), k, pos, rope)
    no(gq.attn_qk_rope, q.transpose(0, 1), k, pos, rope)
    no(gq.attn_qk_rope, q[..., ::2], k[..., ::2], pos, rope)
    no(gq.attn_qk_rope, q, k, pos.long(), rope)
    no(gq.attn_qk_rope, q, k, pos[:7], rope)
    no(gq.attn_qk_rope, q, k, pos[::2], rope)
    no(gq.attn_qk_rope, q, k[:7], pos, rope)
    no(gq.attn_qk_rope, q, k, pos, rope, q_out=q)  # strided
    flat = torch.zeros(8 * 6 * 128 + 8, dtype=torch.bfloat16, device=DEV)
    a, b = flat[:8 * 4 * 128].view(8, 4, 128), flat[8 * 4 * 128:-8].view(8, 2, 128)
    gq.attn_qk_rope(a, b, pos, rope, q_out=a, k_out=b)
    no(gq.attn_qk_rope, a, b, pos, rope, q_out=flat[8:8 + a.numel()].view(8, 4, 128))
    no(gq.attn_qk_rope, a, b, pos, rope, k_out=flat[:b.numel()].view(8, 2, 128))
    no(gq.attn_qk_rope, flat[4:4 + a.numel()].view(8, 4, 128), k, pos, rope)  # alignment
    no(gq.attn_qk_rope, q, k, pos, gq.Rope(rope.inv_freq.double(), HALF))
    no(gq.attn_qk_rope, q, k, pos, gq.Rope(rope.inv_freq, HALF, q_weight=rope.q_weight[:64]))
    no(gq.attn_qk_rope, q, k, pos, gq.Rope(torch.ones(65, device=DEV), HALF))
    no(gq.attn_qk_rope, q, k, pos, gq.Rope(rope.inv_freq, 2))
    no(gq.attn_qk_rope, q, k, pos, gq.Rope(rope.inv_freq, HALF, math.nan))
    no(gq.attn_qk_rope, q, k, pos, gq.Rope(rope.inv_freq, HALF, q_weight=rope.q_weight, eps=0.0))
    no(gq.attn_qk_rope_append, q, k, v, pos, at.int(), cache, rope)
    no(gq.attn_qk_rope_append, q, k, v, pos, at[:7], cache, rope)
    no(gq.attn_qk_rope_append, q, k, q, pos, at, cache, rope)
    no(gq.attn_qk_rope_append, q, k[:, :1], v[:, :1], pos, at, cache, rope)
    assert gq.attn_qk_rope(q[:0], k[:0], pos[:0], rope)[0].shape == (0, 4, 128)
