"""Refusals of the rotary embedding, the cache reads and the shared decode: made on the
host, before any launch, so they need no GPU."""
import ctypes
import math

import pytest
import torch

import gqa_attention_kv_gb300 as gq
from test_capi_host import lib  # noqa: F401
from test_operators_host import BIG, E4, I8, cache, calls, paged_layer  # noqa: F401

FP8 = gq.ATTN_KV_FP8_E4M3
PACK = gq._PACK_ROPE


def rope(inv=4096, rot=128, layout=gq.ATTN_ROPE_HALF, factor=1.0, qw=0, kw=0, eps=1e-6):
    return PACK(inv, rot, layout, factor, qw, kw, eps)


def rope_rc(lib, r=None, q=1 << 20, qs=4096, k=2 << 20, ks=1024, pos=64, n=4, Hq=32, H=8, D=128,  # noqa: F811
            qo=3 << 20, ko=4 << 20):
    return lib.attn_qk_rope(q, qs, k, ks, pos, n, rope() if r is None else r, Hq, H, D, qo, ko,
                            None)


def append_rc(lib, c, r=None, q=1 << 20, qs=4096, k=2 << 20, ks=1024, v=5 << 20, vs=1024, pos=64,  # noqa: F811
              slots=128, n=4, Hq=32, H=8, D=128, qo=3 << 20, ko=4 << 20):
    cs = c.struct()
    return lib.attn_qk_rope_append(q, qs, k, ks, v, vs, pos, slots, n, rope() if r is None else r,
                                   ctypes.byref(cs), Hq, H, D, qo, ko, None, None)


def test_rope_refusals(lib):  # noqa: F811
    null, shape, no, align = (gq.ATTN_ERR_NULL, gq.ATTN_ERR_SHAPE, gq.ATTN_ERR_UNSUPPORTED,
                              gq.ATTN_ERR_ALIGN)
    for bad in (dict(q=None), dict(k=None), dict(pos=None), dict(qo=None), dict(ko=None),
                dict(r=rope(inv=0))):
        assert rope_rc(lib, **bad) == null, bad
    assert lib.attn_qk_rope(16, 0, 16, 0, 64, 4, None, 32, 8, 128, 16, 16, None) == null
    for bad in (dict(n=-1), dict(Hq=0), dict(H=0), dict(qs=4100), dict(qs=4088),
                dict(ks=1016), dict(ks=1028), dict(qs=2 ** 30 + 8), dict(ks=2 ** 40), dict(r=rope(rot=-2)), dict(r=rope(rot=7)),
                dict(r=rope(rot=130)), dict(r=rope(factor=math.inf)), dict(r=rope(factor=math.nan)),
                dict(r=rope(qw=64, eps=0.0)), dict(r=rope(kw=64, eps=math.nan)),
                dict(r=rope(kw=64, eps=1e-31)), dict(r=rope(kw=64, eps=math.inf)),
                # outputs on each other and on inputs, exactly in place only where contiguous
                dict(ko=3 << 20), dict(qo=2 << 20), dict(ko=1 << 20), dict(qo=(1 << 20) + 16),
                dict(ko=(2 << 20) - 16), dict(q=1 << 20, qs=6144, qo=1 << 20)):
        assert rope_rc(lib, **bad) == shape, bad
    for bad in (dict(D=96), dict(r=rope(layout=2)), dict(r=rope(layout=-1))):
        assert rope_rc(lib, **bad) == no, bad
    for bad in (dict(q=(1 << 20) + 8), dict(k=(2 << 20) + 2), dict(qo=(3 << 20) + 4),
                dict(ko=(4 << 20) + 8), dict(r=rope(inv=4098)), dict(r=rope(qw=4097)),
                dict(r=rope(kw=4099))):
        assert rope_rc(lib, **bad) == align, bad
    assert rope_rc(lib, n=0, q=None, k=None) == gq.ATTN_OK
    # eps is looked at where there is a norm only
    assert rope_rc(lib, n=0, r=rope(eps=-1.0)) == gq.ATTN_OK


def test_rope_append_refusals(lib):  # noqa: F811
    big = dict(k=16 << 20, v=32 << 20)
    for bad in (dict(v=None), dict(slots=None), dict(q=None), dict(pos=None)):
        assert append_rc(lib, cache(dtype=gq.ATTN_KV_BF16, **big), **bad) == gq.ATTN_ERR_NULL, bad
    for name in ("k", "v"):
        assert append_rc(lib, cache(dtype=gq.ATTN_KV_BF16, **{**big, name: 0})) == \
            gq.ATTN_ERR_NULL
        assert append_rc(lib, cache(dtype=gq.ATTN_KV_BF16, **{**big, name: (16 << 20) + 8})) == \
            gq.ATTN_ERR_ALIGN
    plain = cache(dtype=gq.ATTN_KV_BF16, **big)
    for bad in (dict(vs=1020), dict(vs=1000), dict(n=-1), dict(qo=5 << 20), dict(ko=(5 << 20) + 16),
                dict(qo=16 << 20), dict(ko=(32 << 20) + 4096)):
        assert append_rc(lib, plain, **bad) == gq.ATTN_ERR_SHAPE, bad
    assert append_rc(lib, plain, D=96) == gq.ATTN_ERR_UNSUPPORTED
    assert append_rc(lib, plain, n=0, q=None) == gq.ATTN_OK
    assert append_rc(lib, cache(dtype=4, **big)) == gq.ATTN_ERR_UNSUPPORTED
    assert append_rc(lib, cache(dtype=FP8, D=64, **big), rope(rot=64), D=64) == \
        gq.ATTN_ERR_UNSUPPORTED
    assert append_rc(lib, cache(dtype=FP8, ref=4100, **big)) == gq.ATTN_ERR_ALIGN
    for dtype in (E4, I8):
        ok = cache(dtype=dtype, **big)
        assert append_rc(lib, ok, ko=None) == gq.ATTN_ERR_NULL
        assert append_rc(lib, ok, vs=2048) == gq.ATTN_ERR_UNSUPPORTED
        assert append_rc(lib, cache(dtype=dtype, sb=24, **big)) == gq.ATTN_ERR_UNSUPPORTED
        assert append_rc(lib, cache(gq.RING, dtype, **big)) == gq.ATTN_ERR_UNSUPPORTED
        assert append_rc(lib, cache(dtype=dtype, ks=None, **big)) == gq.ATTN_ERR_NULL


def read_rc(lib, c, slots=64, n=4, H=8, D=128, ko=1 << 20, vo=2 << 20):  # noqa: F811
    cs = c.struct()
    return lib.attn_kv_read(slots, n, ctypes.byref(cs), H, D, ko, vo, None, None)


def test_read_refusals(lib):  # noqa: F811
    big = dict(k=16 << 20, v=32 << 20)
    plain = cache(dtype=gq.ATTN_KV_BF16, **big)
    for bad in (dict(slots=None), dict(ko=None), dict(vo=None)):
        assert read_rc(lib, plain, **bad) == gq.ATTN_ERR_NULL
    assert lib.attn_kv_read(64, 4, None, 8, 128, 16, 32, None, None) == gq.ATTN_ERR_NULL
    for bad in (dict(n=-1), dict(n=2 ** 31 + 1), dict(H=0), dict(vo=(1 << 20) + 16), dict(ko=16 << 20),
                dict(vo=(32 << 20) + 1024)):
        assert read_rc(lib, plain, **bad) == gq.ATTN_ERR_SHAPE, bad
    for bad in (dict(ko=(1 << 20) + 8), dict(vo=(2 << 20) + 4)):
        assert read_rc(lib, plain, **bad) == gq.ATTN_ERR_ALIGN
    assert read_rc(lib, plain, D=96) == gq.ATTN_ERR_UNSUPPORTED
    assert read_rc(lib, plain, n=0, ko=None) == gq.ATTN_OK
    assert read_rc(lib, cache(dtype=7, **big)) == gq.ATTN_ERR_UNSUPPORTED
    assert read_rc(lib, cache(dtype=FP8, D=64, **big), D=64) == gq.ATTN_ERR_UNSUPPORTED
    assert read_rc(lib, cache(dtype=E4, ref=4100, **big)) == gq.ATTN_ERR_ALIGN
    assert read_rc(lib, cache(dtype=I8, vs=None, **big)) == gq.ATTN_ERR_NULL
    assert read_rc(lib, cache(dtype=E4, sb=48, **big)) == gq.ATTN_ERR_UNSUPPORTED


def shared_rc(lib, c, rows=None, B=2, R=1, L=512, P=256, W=0, Hq=32, H=8, D=128, scale=0.1,  # noqa: F811
              prows=256, plens=512, ws=1 << 20, ws_bytes=BIG, q=1 << 24, out=2 << 24):
    cs = c.struct()
    return lib.attn_decode_shared(q, ctypes.byref(cs), B if rows is None else rows, 64, 128, prows,
                                  plens, B, R, L, P, W, Hq, H, D, scale, out, ws, ws_bytes, None,
                                  None)


def test_shared_refusals(lib):  # noqa: F811
    plain = cache(dtype=gq.ATTN_KV_BF16)
    for bad in (dict(prows=None), dict(plens=None), dict(q=None), dict(out=None), dict(ws=None)):
        assert shared_rc(lib, plain, **bad) == gq.ATTN_ERR_NULL, bad
    for bad in (dict(P=-1), dict(rows=1), dict(rows=3), dict(L=2 ** 31 - 256), dict(B=-1), dict(R=0), dict(L=0),
                dict(scale=0.0), dict(scale=math.nan), dict(Hq=30), dict(out=1 << 24),
                dict(out=(1 << 24) + 16)):
        assert shared_rc(lib, plain, **bad) == gq.ATTN_ERR_SHAPE, bad
    for bad in (dict(q=8), dict(out=40), dict(ws=(1 << 20) + 8)):
        assert shared_rc(lib, plain, **bad) == gq.ATTN_ERR_ALIGN, bad
    for bad in (dict(D=96), dict(Hq=8 * 129)):
        assert shared_rc(lib, plain, **bad) == gq.ATTN_ERR_UNSUPPORTED, bad
    assert shared_rc(lib, cache(gq.RING, gq.ATTN_KV_BF16), W=64) == gq.ATTN_ERR_UNSUPPORTED
    vast = cache(dtype=gq.ATTN_KV_BF16, slots=2 ** 28)  # times 8 heads: 2^31
    assert shared_rc(lib, vast) == gq.ATTN_ERR_UNSUPPORTED
    many = cache(gq.PAGED, gq.ATTN_KV_BF16, sps=0, bs=16)
    assert shared_rc(lib, many, B=4097) == gq.ATTN_ERR_UNSUPPORTED
    need = gq.attn_decode_shared_workspace_size(plain, 2, 1, 32, 512, 256)
    assert shared_rc(lib, plain, ws_bytes=need - 1) == gq.ATTN_ERR_WORKSPACE
    assert shared_rc(lib, plain, B=0, q=None) == gq.ATTN_OK
    for dtype in (E4, I8):
        assert shared_rc(lib, cache(dtype=dtype, ks=None)) == gq.ATTN_ERR_NULL
        assert shared_rc(lib, cache(dtype=dtype, vs=8196)) == gq.ATTN_ERR_ALIGN
        assert shared_rc(lib, cache(dtype=dtype, sb=8)) == gq.ATTN_ERR_UNSUPPORTED
    assert shared_rc(lib, cache(dtype=FP8, D=64), D=64) == gq.ATTN_ERR_UNSUPPORTED
    for bad in (dict(batch=4097), dict(n_q_heads=8 * 129), dict(max_prefix_len=-1)):
        args = dict(batch=2, q_rows=1, n_q_heads=32, max_seq_len=512, max_prefix_len=256)
        with pytest.raises(gq.AttnError):
            gq.attn_decode_shared_workspace_size(many, **{**args, **bad})


@pytest.fixture(autouse=True)
def made_here(monkeypatch):
    """Tensors that the wrappers make: no streams on the CPU."""
    monkeypatch.setattr(gq, "_made", lambda make, like, stream, *args: make(like, *args))


def test_wrappers_refuse_what_the_kernels_would_misread(calls):  # noqa: F811
    """Each in a call that is right otherwise; over CPU tensors, by a library that notes
    what reaches it."""
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    layer = paged_layer()  # 2 heads of 64, 128 slots
    n = 5
    fused = torch.zeros(n, 8, 64, dtype=bf)
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    pos, at = torch.zeros(n, dtype=i32), torch.zeros(n, dtype=i64)
    turn = gq.Rope(torch.ones(32), q_weight=torch.ones(64))

    def no(call, *args, **more):
        before = len(calls)
        with pytest.raises(gq.AttnError):
            call(*args, stream=0, **more)
        assert len(calls) == before

    gq.attn_qk_rope(q, k, pos, turn, stream=0)
    gq.attn_qk_rope_append(q, k, v, pos, at, layer, turn, stream=0)
    gq.attn_kv_read(at, layer, stream=0)
    assert calls == ["attn_qk_rope", "attn_qk_rope_append", "attn_kv_read"]
    for bad in (q.float(), q[:4], q[..., :32], q.transpose(0, 1), q.transpose(1, 2),
                torch.zeros(n, 4, 128, dtype=bf)[..., ::2], q[0]):
        no(gq.attn_qk_rope, bad, k, pos, turn)
        no(gq.attn_qk_rope_append, bad, k, v, pos, at, layer, turn)
    for bad in (k.float(), k[:4], k[:, :, :32], k[:, :1]):
        if bad.shape[1] == 2:
            no(gq.attn_qk_rope, q, bad, pos, turn)
        no(gq.attn_qk_rope_append, q, bad, v, pos, at, layer, turn)
        no(gq.attn_qk_rope_append, q, k, bad, pos, at, layer, turn)
    for bad in (pos.long(), pos[:4], torch.zeros(2 * n, dtype=i32)[::2]):
        no(gq.attn_qk_rope, q, k, bad, turn)
        no(gq.attn_qk_rope_append, q, k, v, bad, at, layer, turn)
    for bad in (at.int(), at[:4], torch.zeros(2 * n, dtype=i64)[::2]):
        no(gq.attn_qk_rope_append, q, k, v, pos, bad, layer, turn)
    no(gq.attn_kv_read, at.int(), layer)
    no(gq.attn_kv_read, torch.zeros(2 * n, dtype=i64)[::2], layer)
    for bad in (torch.zeros(n, 4, 64), torch.zeros(n, 3, 64, dtype=bf), q):
        no(gq.attn_qk_rope, q, k, pos, turn, q_out=bad)
        no(gq.attn_qk_rope_append, q, k, v, pos, at, layer, turn, q_out=bad)
    for bad in (torch.zeros(n, 2, 64), torch.zeros(n + 1, 2, 64, dtype=bf), k):
        no(gq.attn_qk_rope, q, k, pos, turn, k_out=bad)
        no(gq.attn_qk_rope_append, q, k, v, pos, at, layer, turn, k_out=bad)
        no(gq.attn_kv_read, at, layer, k_out=bad)
        no(gq.attn_kv_read, at, layer, v_out=bad)
    for bad in (gq.Rope(torch.ones(32).double()), gq.Rope(torch.ones(64)[::2]),
                gq.Rope(torch.ones(32), k_weight=torch.ones(32)),
                gq.Rope(torch.ones(32), q_weight=torch.ones(64, dtype=bf))):
        no(gq.attn_qk_rope, q, k, pos, bad)
    # a Rope's tensors may be replaced
    turn.q_weight = torch.ones(32)
    no(gq.attn_qk_rope, q, k, pos, turn)
    turn.q_weight = torch.ones(64)
    gq.attn_qk_rope(q, k, pos, turn, stream=0)
    turn.inv_freq.data = torch.ones(16).double()
    no(gq.attn_qk_rope, q, k, pos, turn)
    # reference vectors
    wide = gq.KVCache(gq.LINEAR, torch.zeros(64, 2, 128, dtype=torch.uint8),
                      torch.zeros(64, 2, 128, dtype=torch.uint8), slots_per_seq=64, dtype=FP8,
                      k_ref=torch.zeros(2, 128))
    gq.attn_kv_read(at, wide, stream=0)
    for bad in (torch.zeros(2, 128).double(), torch.zeros(2, 64), torch.zeros(128, 2).T):
        wide.k_ref = bad
        no(gq.attn_kv_read, at, wide)


def test_shared_wrapper_refuses_what_the_kernels_would_misread(calls):  # noqa: F811
    layer = paged_layer()  # 2 rows of 4 pages of 16
    i32 = torch.int32
    good = dict(q=torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16), cache=layer,
                seq_lens=torch.zeros(2, dtype=i32), positions=torch.zeros(2, dtype=i32),
                prefix_rows=torch.zeros(2, dtype=i32), prefix_lens=torch.zeros(2, dtype=i32),
                max_seq_len=64, max_prefix_len=32, window=0, scale=0.1,
                workspace=torch.zeros(64, dtype=torch.uint8), stream=0)
    gq.attn_decode_shared(**good)
    assert calls == ["attn_decode_shared"]
    wrong = dict(q=[torch.zeros(2, 1, 4, 64), torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16),
                    torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16)[:, :, ::2],
                    torch.zeros(3, 1, 4, 64, dtype=torch.bfloat16)])
    for name in ("seq_lens", "positions", "prefix_rows", "prefix_lens"):
        wrong[name] = [torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=i32),
                       torch.zeros(4, dtype=i32)[::2]]
    wrong["workspace"] = [torch.zeros(128, dtype=torch.uint8)[::2]]
    wrong["out"] = [torch.zeros(2, 1, 4, 64), torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)]
    for name, values in wrong.items():
        for bad in values:
            with pytest.raises(gq.AttnError):
                gq.attn_decode_shared(**{**good, name: bad})
    assert calls == ["attn_decode_shared"]


def test_rope_frequencies():
    """The formulas, at their ends and between."""
    inv, times = gq.rope_frequencies(64, 10000.0)
    want = 10000.0 ** (-torch.arange(32).double() / 32)
    assert torch.equal(inv, want.float()) and times == 1.0
    linear, _ = gq.rope_frequencies(64, 10000.0, "linear", 4.0)
    assert torch.equal(linear, (want / 4).float())
    ntk, _ = gq.rope_frequencies(64, 10000.0, "ntk", 4.0)
    assert ntk[0] == 1.0 and abs(ntk[-1].item() / (want[-1].item() / 4) - 1) < 1e-6
    yarn, times = gq.rope_frequencies(64, 10000.0, "yarn", 4.0, 4096)
    assert times == 0.1 * math.log(4.0) + 1
    turns = 4096 * want / (2 * math.pi)
    assert torch.equal(yarn[turns > 32 * 1.4], want.float()[turns > 32 * 1.4])
    assert torch.equal(yarn[turns < 1 / 1.4], (want / 4).float()[turns < 1 / 1.4])
    ratio = yarn.double() / want
    assert (ratio.diff() <= 1e-6).all() and ratio.min() >= 0.25 - 1e-6 and ratio.max() <= 1 + 1e-6
    assert gq.rope_frequencies(0)[0].numel() == 0
    for bad in (dict(rot_dim=7), dict(rot_dim=-2), dict(rot_dim=8, base=1.0),
                dict(rot_dim=8, scaling="other"), dict(rot_dim=8, scaling="linear", factor=0.0),
                dict(rot_dim=2, scaling="ntk"), dict(rot_dim=8, scaling="yarn", factor=2.0),
                dict(rot_dim=8, scaling="yarn", factor=0.5, original_len=100)):
        with pytest.raises(gq.AttnError):
            gq.rope_frequencies(**bad)
