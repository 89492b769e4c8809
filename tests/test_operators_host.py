"""Refusals of the scaled caches, the windows with sinks and the page
operations: made on the host, before any launch, so they need no GPU."""
import ctypes

import pytest

import gqa_attention_kv_gb300 as gq
from test_capi_host import FakeTensor, lib  # noqa: F401

E4, I8 = gq.ATTN_KV_FP8_E4M3_SCALED, gq.ATTN_KV_INT8_SCALED
BIG = 1 << 30


def cache(kind=gq.LINEAR, dtype=E4, slots=1024, sps=512, bs=0, sb=16, D=128, Hkv=8, ks=4096,
          vs=8192, layout=gq.ATTN_LAYOUT_BSHD, blocks=64, k=4096, v=8192, ref=None):
    per = bs if kind == gq.PAGED else sps
    shape = (slots, Hkv, D) if layout == gq.ATTN_LAYOUT_BSHD else (slots // per, Hkv, per, D)
    fake = lambda a: None if a is None else FakeTensor(a, (1,))  # noqa: E731
    return gq.KVCache(kind, FakeTensor(k, shape), FakeTensor(v, shape), slots_per_seq=sps,
                      block_table=FakeTensor(1 << 20, (2, blocks)) if kind == gq.PAGED else None,
                      block_size=bs, dtype=dtype, layout=layout, k_scale=fake(ks),
                      v_scale=fake(vs), scale_block=sb, k_ref=fake(ref))


def append_rc(lib, c, n=4, D=128):
    return lib.attn_kv_append(16, 32, 64, n, ctypes.byref(c.struct()), 8, D, None, None)


def decode_rc(lib, c, W=0, S=None, B=2, R=1, L=512, D=128, ws=1 << 20, ws_bytes=BIG, scale=0.1):
    cs = c.struct()
    if S is None:
        return lib.attn_decode(16, ctypes.byref(cs), 64, 128, B, R, L, W, 32, 8, D, scale, 32, ws,
                               ws_bytes, None, None)
    return lib.attn_decode_sinks(16, ctypes.byref(cs), 64, 128, B, R, L, W, S, 32, 8, D, scale, 32,
                                 ws, ws_bytes, None, None)


@pytest.mark.parametrize("dtype", [E4, I8])
def test_scaled_cache_refusals(lib, dtype):  # noqa: F811
    for rc in (append_rc, decode_rc):
        assert rc(lib, cache(dtype=dtype, sb=24)) == gq.ATTN_ERR_UNSUPPORTED
        assert rc(lib, cache(dtype=dtype, sb=0)) == gq.ATTN_ERR_UNSUPPORTED
        assert rc(lib, cache(dtype=dtype, sb=256)) == gq.ATTN_ERR_UNSUPPORTED
        # whole blocks in a request's slots, a page and the cache
        assert rc(lib, cache(dtype=dtype, sps=504)) == gq.ATTN_ERR_SHAPE
        assert rc(lib, cache(gq.PAGED, dtype, sps=0, bs=8)) == gq.ATTN_ERR_SHAPE
        assert rc(lib, cache(gq.PAGED, dtype, sps=0, bs=16, sb=32)) == gq.ATTN_ERR_SHAPE
        assert rc(lib, cache(dtype=dtype, slots=1032)) == gq.ATTN_ERR_SHAPE
        assert rc(lib, cache(dtype=dtype, ks=None)) == gq.ATTN_ERR_NULL
        assert rc(lib, cache(dtype=dtype, vs=None)) == gq.ATTN_ERR_NULL
        assert rc(lib, cache(dtype=dtype, vs=8196)) == gq.ATTN_ERR_ALIGN
        assert rc(lib, cache(dtype=dtype, k=4100)) == gq.ATTN_ERR_ALIGN
        assert rc(lib, cache(dtype=dtype), D=96) == gq.ATTN_ERR_UNSUPPORTED
    assert append_rc(lib, cache(dtype=dtype, ref=4100)) == gq.ATTN_ERR_ALIGN
    ring = cache(gq.RING, dtype)
    assert append_rc(lib, ring) == gq.ATTN_ERR_UNSUPPORTED
    assert decode_rc(lib, ring, W=64) == gq.ATTN_ERR_UNSUPPORTED
    assert append_rc(lib, cache(dtype=dtype), n=0) == gq.ATTN_OK
    assert append_rc(lib, cache(dtype=4)) == gq.ATTN_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", [E4, I8])
def test_scaled_decode_refusals(lib, dtype):  # noqa: F811
    c = cache(dtype=dtype)
    cs = c.struct()
    need = lib.attn_decode_workspace_size(ctypes.byref(cs), 2, 1, 32, 8, 128, 512, 0)
    assert 0 < need < BIG
    assert decode_rc(lib, c, ws=None, ws_bytes=0) == gq.ATTN_ERR_NULL
    assert decode_rc(lib, c, ws_bytes=need - 1) == gq.ATTN_ERR_WORKSPACE
    assert decode_rc(lib, c, ws=(1 << 20) + 8) == gq.ATTN_ERR_ALIGN
    assert decode_rc(lib, c, scale=float("nan")) == gq.ATTN_ERR_SHAPE
    assert decode_rc(lib, c, B=0) == gq.ATTN_OK
    args = (2, 1, 512, 0, 32, 8, 128, 0.1, 32)
    assert lib.attn_decode_noalloc(16, ctypes.byref(cs), 64, 128, *args, None,
                                   None) == gq.ATTN_ERR_UNSUPPORTED
    # the fused step: no rotary embedding, a workspace before anything is appended
    step = lambda rope, ws: lib.attn_decode_append(  # noqa: E731
        16, 32, 48, 64, rope, ctypes.byref(cs), 64, 128, *args, ws, BIG, None, 0, None)
    assert step(4096, 1 << 20) == gq.ATTN_ERR_UNSUPPORTED
    assert step(None, None) == gq.ATTN_ERR_NULL
    assert gq.attn_decode_kernel_launches(c, 2, 1, 32, 512) in (1, 2)
    assert gq.attn_decode_kernel_launches(c, 2, 1, 32, 512, with_append=True) == 1 + \
        gq.attn_decode_kernel_launches(c, 2, 1, 32, 512)
    with pytest.raises(gq.AttnError):
        gq.attn_decode_kernel_launches(c, 2, 1, 32, 512, with_append=True, with_rope=True)


def test_sinks_refusals(lib):  # noqa: F811
    bf = lambda kind=gq.LINEAR, **kw: cache(kind, gq.ATTN_KV_BF16, **kw)  # noqa: E731
    assert decode_rc(lib, bf(), W=64, S=-1) == gq.ATTN_ERR_SHAPE
    # a ring holds the sinks beside the window
    assert decode_rc(lib, bf(gq.RING), W=500, S=13) == gq.ATTN_ERR_SHAPE
    assert decode_rc(lib, bf(gq.RING), W=500, S=12, R=2) == gq.ATTN_ERR_SHAPE
    assert decode_rc(lib, bf(gq.RING), W=500, S=12, ws_bytes=8) == gq.ATTN_ERR_WORKSPACE
    assert decode_rc(lib, bf(gq.RING), W=0, S=4) == gq.ATTN_ERR_SHAPE
    assert decode_rc(lib, bf(), W=64, S=4, ws=None) == gq.ATTN_ERR_NULL
    assert decode_rc(lib, bf(k=4104), W=64, S=4) == gq.ATTN_ERR_ALIGN
    assert decode_rc(lib, bf(), W=64, S=4, D=96) == gq.ATTN_ERR_UNSUPPORTED
    assert decode_rc(lib, bf(), W=64, S=4, scale=-1.0) == gq.ATTN_ERR_SHAPE
    assert decode_rc(lib, bf(), W=64, S=4, L=0) == gq.ATTN_ERR_SHAPE
    assert decode_rc(lib, bf(gq.PAGED, sps=0, bs=8, blocks=8), W=64, S=4) == gq.ATTN_ERR_SHAPE
    assert decode_rc(lib, cache(dtype=gq.ATTN_KV_FP8_E4M3, D=64), W=8, S=1,
                     D=64) == gq.ATTN_ERR_UNSUPPORTED
    assert decode_rc(lib, cache(gq.RING, I8), W=64, S=4) == gq.ATTN_ERR_UNSUPPORTED
    cs = bf().struct()
    size = lib.attn_decode_sinks_workspace_size
    assert size(ctypes.byref(cs), 2, 1, 32, 8, 128, 512, 64, -1) == ctypes.c_size_t(-1).value
    assert size(ctypes.byref(cs), 0, 1, 32, 8, 128, 512, 64, 4) == 0
    pre = lambda S, Hq=8, q=16: lib.attn_prefill_sinks(  # noqa: E731
        q, 32, 48, 1, 64, 16, S, Hq, 4, 64, 0.1, 64, None, None)
    assert pre(-1) == gq.ATTN_ERR_SHAPE
    assert pre(4, Hq=6) == gq.ATTN_ERR_SHAPE
    assert pre(4, q=None) == gq.ATTN_ERR_NULL
    assert pre(4, q=24) == gq.ATTN_ERR_ALIGN


def test_page_operation_refusals(lib):  # noqa: F811
    for f in (lib.attn_pages_free, lib.attn_pages_reserve):
        assert f(16, 8, 4, 4, 4, 4, 2, None, 64, None, None) == gq.ATTN_ERR_NULL
        assert f(None, 8, 4, 4, 4, 4, 2, 16, 64, None, None) == gq.ATTN_ERR_NULL
        assert f(16, 0, 4, 4, 4, 4, 2, 16, 64, None, None) == gq.ATTN_ERR_SHAPE
        assert f(16, 8, 4, 4, 4, 4, -1, 16, 64, None, None) == gq.ATTN_ERR_SHAPE
        assert f(16, 8, 4, 4, 4, 4, 2, 16, 0, None, None) == gq.ATTN_ERR_SHAPE
        assert f(16, 8, 4, None, 4, 4, 2, 16, 64, None, None) == gq.ATTN_ERR_NULL
        assert f(16, 8, 4, 4, 4, 4, 2, 20, 64, None, None) == gq.ATTN_ERR_ALIGN
        assert f(16, 8, 4, None, None, None, 0, 16, 64, None, None) == gq.ATTN_OK
    fork = lambda n=2, bs=16, most=2, moves=16, count=16: lib.attn_pages_fork(  # noqa: E731
        16, 8, 4, 4, 4, 4, n, bs, 16, 64, moves, most, count, None, None)
    assert fork(n=-1) == gq.ATTN_ERR_SHAPE
    assert fork(bs=0) == gq.ATTN_ERR_SHAPE
    assert fork(most=1) == gq.ATTN_ERR_SHAPE
    assert fork(moves=None) == gq.ATTN_ERR_NULL
    assert fork(count=None) == gq.ATTN_ERR_NULL
    need = lib.attn_pages_workspace_size(64)
    assert lib.attn_pages_workspace_size(0) == ctypes.c_size_t(-1).value
    compact = lambda bs=16, most=2, moves=16, used=16, ws=16, size=need: (  # noqa: E731
        lib.attn_pages_compact(16, 8, 4, bs, 16, 64, moves, most, 16, used, ws, size, None, None))
    assert compact(bs=0) == gq.ATTN_ERR_SHAPE
    assert compact(most=-1) == gq.ATTN_ERR_SHAPE
    assert compact(moves=None) == gq.ATTN_ERR_NULL
    assert compact(used=None) == gq.ATTN_ERR_NULL
    assert compact(ws=None) == gq.ATTN_ERR_NULL
    assert compact(size=need - 1) == gq.ATTN_ERR_WORKSPACE
    assert compact(ws=24) == gq.ATTN_ERR_ALIGN


def test_page_copy_refusals(lib):  # noqa: F811
    def rc(caches, D=128, moves=16, count=16, most=4, n=None):
        arr = (gq._Cache * len(caches))(*[c.struct() for c in caches])
        return lib.attn_pages_copy(arr, len(caches) if n is None else n, 8, D, moves, count, most,
                                   None, None)

    paged = lambda **kw: cache(gq.PAGED, kw.pop("dtype", I8), sps=0, bs=kw.pop("bs", 32),  # noqa: E731
                               **kw)
    assert rc([cache()]) == gq.ATTN_ERR_UNSUPPORTED                  # not paged
    assert rc([paged()], D=80) == gq.ATTN_ERR_UNSUPPORTED
    assert rc([paged(dtype=9)]) == gq.ATTN_ERR_UNSUPPORTED
    assert rc([paged(ks=None)]) == gq.ATTN_ERR_NULL
    assert rc([paged(k=20)]) == gq.ATTN_ERR_ALIGN
    assert rc([paged(), paged(bs=64)]) == gq.ATTN_ERR_SHAPE          # layers alike
    assert rc([paged(), paged(dtype=E4)]) == gq.ATTN_ERR_SHAPE
    assert rc([paged(), paged(sb=32)]) == gq.ATTN_ERR_SHAPE
    assert rc([paged(), paged(slots=2048)]) == gq.ATTN_ERR_SHAPE
    assert rc([paged()], moves=None) == gq.ATTN_ERR_NULL
    assert rc([paged()], count=None) == gq.ATTN_ERR_NULL
    assert rc([paged()], most=-1) == gq.ATTN_ERR_SHAPE
    assert rc([paged()], most=0) == gq.ATTN_OK
    assert rc([paged()], n=0) == gq.ATTN_OK
    assert "free page" in gq.attn_status_string(gq.ATTN_ERR_PAGES)


def test_wrappers_refuse_what_the_kernels_would_misread():
    """Tensors of another type, order or device, and shapes that disagree."""
    import torch

    bad = torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16)  # not on a GPU
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises((gq.AttnError, RuntimeError)):
        gq.attn_decode_sinks(bad, cache(dtype=gq.ATTN_KV_BF16, D=64), i32, i32, 16, 8, 4, 0.1)
    with pytest.raises((gq.AttnError, RuntimeError)):
        gq.attn_prefill_sinks(bad, bad, bad, 8, 4, 0.1)
    with pytest.raises((gq.AttnError, RuntimeError)):
        gq.attn_pages_free(i32.view(1, 2), i32, i32, i32, i32)
    codes, scale = torch.zeros(64, 2, 64, dtype=torch.int8), torch.ones(4, 2)
    gq.KVCache(gq.LINEAR, codes, codes, slots_per_seq=64, dtype=I8, k_scale=scale, v_scale=scale,
               scale_block=16)
    for other in (torch.ones(2, 4).T, torch.ones(2, 2), torch.ones(4, 2).double()):
        with pytest.raises(gq.AttnError):
            gq.KVCache(gq.LINEAR, codes, codes, slots_per_seq=64, dtype=I8, k_scale=scale,
                       v_scale=other, scale_block=16)


@pytest.fixture
def calls(monkeypatch):
    """The wrappers over CPU tensors, with a library that notes what reaches it."""
    import torch

    class Library:
        def __init__(self):
            self.names = []

        def __getattr__(self, name):
            return lambda *args: self.names.append(name) or 0

    fake = Library()
    monkeypatch.setattr(gq, "lib", lambda: fake)
    monkeypatch.setattr(gq, "attn_status_string", lambda status: "")
    monkeypatch.setattr(gq, "_device", lambda: torch.zeros(0).get_device())  # -1: the CPU's
    return fake.names


def paged_layer(pages=8, H=2, D=64, dtype=gq.ATTN_KV_BF16):
    import torch

    store = {gq.ATTN_KV_BF16: torch.bfloat16, I8: torch.int8}.get(dtype, torch.uint8)
    more = {}
    if dtype in (E4, I8):
        more = dict(scale_block=16, k_scale=torch.zeros(pages, H), v_scale=torch.zeros(pages, H))
    return gq.KVCache(gq.PAGED, torch.zeros(pages * 16, H, D, dtype=store),
                      torch.zeros(pages * 16, H, D, dtype=store), block_size=16,
                      block_table=torch.zeros(2, 4, dtype=torch.int32), dtype=dtype, **more)


@pytest.mark.parametrize("dtype", [gq.ATTN_KV_BF16, gq.ATTN_KV_FP8_E4M3, E4, I8])
@pytest.mark.parametrize("name", ["k", "v"])
def test_page_copies_look_at_tensors_that_were_replaced(calls, dtype, name):
    """k and v of a layer may be replaced; the others' place then no longer tells theirs."""
    import torch

    moves, count = torch.zeros(3, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    layers = [paged_layer(dtype=dtype) for _ in range(3)]
    copy = lambda: gq.attn_pages_copy(layers, moves, count, stream=0)  # noqa: E731
    copy()
    for at in (0, 2):                      # the first layer's larger, a later one's smaller
        old = getattr(layers[at], name)
        new = torch.zeros(old.shape[0] * 2 if at == 0 else 16, *old.shape[1:], dtype=old.dtype)
        setattr(layers[at], name, new)
        with pytest.raises(gq.AttnError):
            copy()
        setattr(layers[at], name, old.clone())
        copy()
        getattr(layers[at], name).data = new   # the tensor itself made another
        with pytest.raises(gq.AttnError):
            copy()
        setattr(layers[at], name, old)
    for bad in (torch.zeros(128, 2, 128, dtype=old.dtype)[..., :64],
                torch.zeros(128, 2, 64, dtype=torch.float32), old.view(128, 1, 128)):
        setattr(layers[1], name, bad)
        with pytest.raises(gq.AttnError):
            copy()
    setattr(layers[1], name, old)
    if dtype in (E4, I8):
        layers[1].k_scale = torch.zeros(4, 2)
        with pytest.raises(gq.AttnError):
            copy()
        layers[1].k_scale = torch.zeros(8, 2)
    copy()
    assert calls == ["attn_pages_copy"] * 4


def test_scaled_caches_and_sinks_refuse_what_the_kernels_would_misread(calls):
    """Tensors of another type, size, order or device, each in a call that is right
    without it; nothing reaches the library."""
    import torch

    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    B, R, Hq, H, D = 2, 3, 4, 2, 64
    z = torch.zeros
    good = {"q": z(B, R, Hq, D, dtype=bf), "k_new": z(B * R, H, D, dtype=bf),
            "v_new": z(B * R, H, D, dtype=bf), "slots": z(B * R, dtype=i64),
            "lens": z(B, dtype=i32), "pos": z(B * R, dtype=i32), "ws": z(64, dtype=torch.uint8),
            "out": z(B, R, Hq, D, dtype=bf)}

    def append(c, a):
        gq.attn_kv_append(a["k_new"], a["v_new"], a["slots"], c, stream=0)

    def decode(c, a):
        gq.attn_decode(a["q"], c, a["lens"], a["pos"], 64, 0, 0.1, out=a["out"],
                       workspace=a["ws"], stream=0)

    def sinks(c, a):
        gq.attn_decode_sinks(a["q"], c, a["lens"], a["pos"], 64, 8, 2, 0.1, out=a["out"],
                             workspace=a["ws"], stream=0)

    def step(c, a):
        gq.attn_decode_append(a["q"], a["k_new"], a["v_new"], a["slots"], c, a["lens"], a["pos"],
                              64, 0, 0.1, out=a["out"], workspace=a["ws"], stream=0)

    rows = {"k_new": [z(B * R - 1, H, D, dtype=bf), z(B * R, H, D), z(B * R, H, 2 * D, dtype=bf),
                      z(H, B * R, D, dtype=bf).transpose(0, 1)],
            "v_new": [z(1, H, D, dtype=bf)],
            "slots": [z(B * R, dtype=i32), z(2 * B * R, dtype=i64)[::2]]}
    reads = {"q": [z(B, R, Hq, D), z(B, R, Hq, 2 * D, dtype=bf),
                   z(B, Hq, R, D, dtype=bf).transpose(1, 2)],
             "out": [z(B, R, Hq, D), z(B, R, 1, D, dtype=bf)],
             "lens": [z(B, dtype=i64), z(1, dtype=i32)],
             "pos": [z(B * R, dtype=i64), z(B * R - 1, dtype=i32), z(2 * B * R, dtype=i32)[::2]],
             "ws": [z(2, 64, dtype=torch.uint8)[:, ::2]]}
    fields = {"k": [z(128, H, D), z(64, H, D, dtype=torch.int8), z(128, H, D, dtype=bf)],
              "v": [z(8, H, D, dtype=torch.int8)],
              "k_scale": [z(7, H), z(8, H).double()], "v_scale": [z(4, 2 * H), None],
              "block_table": [z(2, 4, dtype=i64), z(1, 4, dtype=i32), z(8, dtype=i32)]}
    single = paged_layer()
    single.block_table = z(4, dtype=i32)           # a request's row by itself
    sinks(single, {**good, "q": good["q"][:1], "out": good["out"][:1]})
    table = {append: rows, decode: reads, sinks: reads, step: {**rows, **reads}}
    for call, arguments in table.items():
        for dtype in (E4, I8) + ((gq.ATTN_KV_BF16,) if call is sinks else ()):
            del calls[:]
            call(paged_layer(dtype=dtype), good)
            assert len(calls) == 1
            for name, bad in arguments.items():
                for x in bad:
                    with pytest.raises(gq.AttnError):
                        call(paged_layer(dtype=dtype), {**good, name: x})
            for name, bad in fields.items():
                if (name == "block_table" and call is append) or \
                        (name.endswith("scale") and dtype == gq.ATTN_KV_BF16):
                    continue
                for x in bad:
                    if x is not None and x.dtype is bf and dtype == gq.ATTN_KV_BF16:
                        continue
                    layer = paged_layer(dtype=dtype)
                    setattr(layer, name, x)
                    with pytest.raises(gq.AttnError):
                        call(layer, good)
            if call is append:
                layer = paged_layer(dtype=dtype)
                for x in (z(H, D).double(), z(H, 2 * D)[:, ::2], z(1, D)):
                    layer.k_ref = x
                    with pytest.raises(gq.AttnError):
                        call(layer, good)
            assert len(calls) == 1


def test_a_scaled_cache_has_both_scales(calls):
    import torch

    codes, scale = torch.zeros(64, 2, 64, dtype=torch.int8), torch.ones(4, 2)
    for k_scale, v_scale in ((scale, None), (None, scale)):
        with pytest.raises(gq.AttnError):
            gq.KVCache(gq.LINEAR, codes, codes, slots_per_seq=64, dtype=I8, k_scale=k_scale,
                       v_scale=v_scale, scale_block=16)


def test_sinks_and_page_wrappers_refuse_what_the_kernels_would_misread(calls, monkeypatch):
    """Types, order, device and shapes, each in a call that is right without it."""
    import torch

    i32, z = torch.int32, torch.zeros
    ints = lambda *shape: z(*shape, dtype=i32)  # noqa: E731
    table, refs, rows, moves, one = ints(4, 6), ints(32), ints(3), ints(8, 3), ints(1)
    space = z(4096, dtype=torch.uint8)
    q, k = z(2, 5, 4, 64, dtype=torch.bfloat16), z(2, 5, 2, 64, dtype=torch.bfloat16)
    cases = [
        (lambda a, b, c, d, e: gq.attn_pages_free(a, b, c, d, e, stream=0),
         [table, refs, rows, rows, rows]),
        (lambda a, b, c, d, e: gq.attn_pages_reserve(a, b, c, d, e, stream=0),
         [table, refs, rows, rows, rows]),
        (lambda a, b, c, d, e, m, n: gq.attn_pages_fork(a, b, c, d, e, 16, m, n, stream=0),
         [table, refs, rows, rows, rows, moves, one]),
        (lambda a, b, m, n, u: gq.attn_pages_compact(a, b, 16, m, n, u, workspace=space, stream=0),
         [table, refs, moves, one, one]),
        (lambda m, n: gq.attn_pages_copy([], m, n, stream=0), [moves, one]),
        (lambda a, b, c: gq.attn_prefill_sinks(a, b, c, 8, 4, 0.1, out=q, stream=0),
         [q, k, k]),
    ]
    for call, good in cases:
        del calls[:]
        call(*good)
        assert len(calls) == 1
        for at, x in enumerate(good):
            wide = torch.cat([x, x], -1)
            bad = [x.double(), wide[..., ::2]]
            if x.dim() > 1:
                bad.append(x[..., :-1].contiguous() if x is not table else x[0])
            for y in bad:
                if wide[..., ::2].is_contiguous() and y is bad[1]:
                    continue
                with pytest.raises(gq.AttnError):
                    call(*good[:at], y, *good[at + 1:])
        assert len(calls) == 1
    with pytest.raises(gq.AttnError):
        gq.attn_pages_compact(table, refs, 16, moves, one, one, workspace=z(9, 9)[:, ::2], stream=0)
    for call, good in cases[:3]:               # row arguments of one length
        with pytest.raises(gq.AttnError):
            call(*good[:4], ints(2), *good[5:])
    monkeypatch.setattr(gq, "_device", lambda: 0)
    for call, good in cases:                   # these tensors are the CPU's
        with pytest.raises(gq.AttnError):
            call(*good)
    assert len(calls) == 1
