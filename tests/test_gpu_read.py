"""Cache slots read back as bf16 rows."""
import pytest
import torch

import gqa_attention_kv_gb300 as gq
import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPE = {"bf16": gq.ATTN_KV_BF16, "fp8": gq.ATTN_KV_FP8_E4M3,
         "e4m3": gq.ATTN_KV_FP8_E4M3_SCALED, "int8": gq.ATTN_KV_INT8_SCALED}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def build(fmt, slots, H, D, sb, per, head_major, with_ref, seed):
    g = gen(seed)
    scaled = fmt in ("e4m3", "int8")
    if fmt == "bf16":
        k, v = (torch.randn(slots, H, D, generator=g).bfloat16() for _ in range(2))
    elif fmt == "int8":
        k, v = (torch.randint(-127, 128, (slots, H, D), generator=g).to(torch.int8)
                for _ in range(2))
    else:  # every code but the NaNs
        k, v = (torch.randint(0, 127, (slots, H, D), generator=g).to(torch.uint8) |
                (torch.randint(0, 2, (slots, H, D), generator=g) * 128).to(torch.uint8)
                for _ in range(2))
    ks, vs = (torch.exp(torch.randn(slots // sb, H, generator=g) * 8) for _ in range(2))
    k_ref = torch.randn(H, D, generator=g) if with_ref and fmt != "bf16" else None
    values = []
    for x, s in ((k, ks), (v, vs)):
        if fmt == "bf16":
            values.append(x.double())
        elif scaled:
            values.append(ref.dequantized(fmt, x, s, sb))
        else:
            values.append(ref.code_values("e4m3", x))
    lay = lambda x: x if not head_major else \
        x.view(-1, per, H, D).transpose(1, 2).contiguous()  # noqa: E731
    more = dict(k_scale=ks.to(DEV), v_scale=vs.to(DEV), scale_block=sb) if scaled else {}
    cache = gq.KVCache(gq.LINEAR, lay(k).to(DEV), lay(v).to(DEV), slots_per_seq=per,
                       dtype=DTYPE[fmt], k_ref=None if k_ref is None else k_ref.to(DEV),
                       layout=gq.ATTN_LAYOUT_BHSD if head_major else gq.ATTN_LAYOUT_BSHD, **more)
    return cache, values, k_ref


@pytest.mark.parametrize("fmt,D,H,sb,head_major,with_ref,n", [
    ("bf16", 64, 3, 16, False, False, 77), ("bf16", 128, 8, 16, True, False, 300),
    ("fp8", 128, 4, 16, False, True, 200), ("fp8", 128, 1, 16, True, False, 1),
    ("e4m3", 128, 8, 16, False, False, 500), ("e4m3", 64, 5, 32, True, True, 130),
    ("int8", 128, 4, 64, False, True, 3000), ("int8", 64, 2, 128, True, False, 40),
    ("int8", 64, 40, 16, False, False, 9)])
def test_read(fmt, D, H, sb, head_major, with_ref, n):
    slots, per = 512, 128
    cache, (kd, vd), k_ref = build(fmt, slots, H, D, sb, per, head_major, with_ref, n)
    at = torch.randint(0, slots, (n,), generator=gen(n))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k, v = gq.attn_kv_read(at.to(DEV), cache, err=err)
    assert int(err) == 0
    if fmt == "bf16":
        assert torch.equal(k.cpu().double(), kd[at]) and torch.equal(v.cpu().double(), vd[at])
        return
    # one rounding to float32 (half a step, 2^-24, of the sum's larger term) and one to bf16
    big = kd[at].abs() + (0 if k_ref is None else k_ref.double().abs())
    want = kd[at] + (0 if k_ref is None else k_ref.double())
    assert ((k.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -23 * big).all()
    assert ((v.cpu().double() - vd[at]).abs() <= (2.0 ** -8 + 2.0 ** -23) * vd[at].abs()).all()


def test_slots_outside_give_zeros():
    cache, (kd, vd), _ = build("e4m3", 64, 2, 64, 16, 64, False, False, 1)
    at = torch.tensor([3, -1, 64, 63, 2 ** 40, -2 ** 40])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k, v = gq.attn_kv_read(at.to(DEV), cache, err=err)
    assert int(err) == gq.ATTN_ERR_BOUNDS
    for x in (k, v):
        assert x[[0, 3]].any() and not x[[1, 2, 4, 5]].any()


def test_what_is_not_finite_and_small_scales():
    k = torch.tensor([0x7F, 0xFF, 0x7E, 0x01], dtype=torch.uint8).repeat(16, 1, 16)
    ks = torch.tensor([[0.0]])
    cache = gq.KVCache(gq.LINEAR, k.to(DEV), k.to(DEV), slots_per_seq=16,
                       dtype=gq.ATTN_KV_FP8_E4M3_SCALED, k_scale=ks.to(DEV),
                       v_scale=torch.tensor([[3.0e38]], device=DEV), scale_block=16)
    a, b = gq.attn_kv_read(torch.tensor([5], device=DEV), cache)
    assert torch.isnan(a[0, 0, 0]) and torch.isnan(a[0, 0, 1])
    assert a[0, 0, 2].item() == 448 * 2.0 ** -64 and a[0, 0, 3].item() == 2.0 ** -73
    assert b[0, 0, 2].item() == float("inf") and torch.isfinite(b[0, 0, 3])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_read_gives_back_what_append_wrote(fmt):
    """Within half a step of the codes: 2^-4 of a value or the smallest code's half
    (E4M3), half a step of the block's scale (INT8)."""
    g = gen(3)
    n, H, D = 100, 2, 128
    k, v = (torch.randn(n, H, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    raw = torch.uint8 if fmt == "e4m3" else torch.int8
    cache = gq.KVCache(gq.LINEAR, torch.zeros(112, H, D, dtype=raw, device=DEV),
                       torch.zeros(112, H, D, dtype=raw, device=DEV), slots_per_seq=112,
                       dtype=DTYPE[fmt], k_scale=torch.zeros(7, H, device=DEV),
                       v_scale=torch.zeros(7, H, device=DEV), scale_block=16)
    at = torch.arange(n, device=DEV)
    gq.attn_kv_append(k, v, at, cache)
    for new, got, s in zip((k, v), gq.attn_kv_read(at, cache), (cache.k_scale, cache.v_scale)):
        s = s[at // 16][..., None].double()
        x = new.double()
        step = torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s) if fmt == "e4m3" else 0.5 * s
        assert ((got.double() - x).abs() <= step * (1 + 2.0 ** -20) + 2.0 ** -8 * got.double().abs()).all()


def test_stream_graph_and_refusals():
    cache, _, _ = build("int8", 256, 2, 128, 16, 256, False, False, 8)
    at = torch.arange(50, device=DEV)
    k, v = gq.attn_kv_read(at, cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ks, vs = gq.attn_kv_read(at, cache, stream=s)
    s.synchronize()
    assert torch.equal(k, ks) and torch.equal(v, vs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq.attn_kv_read(at, cache, k_out=ks, v_out=vs)
    at.add_(100)
    graph.replay()
    k, v = gq.attn_kv_read(at, cache)
    assert torch.equal(k, ks) and torch.equal(v, vs)

    def no(*a, **kw):
        with pytest.raises(gq.AttnError):
            gq.attn_kv_read(*a, **kw)

    no(at.int(), cache)
    no(at.cpu(), cache)
    no(at[::2], cache)
    no(at, cache, k_out=ks.float())
    no(at, cache, k_out=ks[:49])
    no(at, cache, k_out=vs, v_out=vs)
    no(at, cache, k_out=cache.k.view(torch.bfloat16).view(-1)[:ks.numel()].view(ks.shape))
    assert gq.attn_kv_read(at[:0], cache)[0].shape == (0, 2, 128)


def test_offsets_past_32_bits():
    """A slot whose bytes lie past 2^32 from the cache's start."""
    H, D = 8, 128
    slots = (1 << 31) // (H * D) + 100
    k = torch.zeros(slots, H, D, dtype=torch.bfloat16, device=DEV)
    cache = gq.KVCache(gq.LINEAR, k, k, slots_per_seq=slots)
    k[slots - 3] = 2.5
    a, b = gq.attn_kv_read(torch.tensor([slots - 3, 0], device=DEV), cache)
    assert (a[0] == 2.5).all() and not a[1].any() and torch.equal(a, b)
