"""Page operations against plain loops, and the operators in one serving run."""
import pytest
import torch

import gqa_attention_kv_gb300 as gq
import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def filled(g, rows, width, pages, used, share=0.2):
    """A table with `used` entries a row dealt from a shuffled pool, some shared."""
    table = torch.full((rows, width), -1, dtype=torch.int32)
    deck = torch.randperm(pages, generator=g).tolist()
    for r in range(rows):
        for j in range(used[r]):
            if r and j < used[r - 1] and torch.rand((), generator=g) < share:
                table[r, j] = table[r - 1, j]
            else:
                table[r, j] = deck.pop()
    refs = torch.zeros(pages, dtype=torch.int32)
    for p in table[table >= 0].tolist():
        refs[p] += 1
    return table, refs


def error():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def same(cpu, gpu):
    torch.cuda.synchronize()
    assert torch.equal(cpu, gpu.cpu())


@pytest.mark.parametrize("rows,width,pages", [(1, 1, 1), (5, 9, 60), (40, 300, 9000),
                                              (1500, 3, 5001)])
def test_free_and_reserve(rows, width, pages):
    g = gen(rows)
    used = torch.randint(0, width + 1, (rows,), generator=g).tolist()
    used = [min(u, (pages * 2 // 3) // rows) for u in used]
    table, refs = filled(g, rows, width, pages, used)
    t, r, err = table.to(DEV), refs.to(DEV), error()
    which = torch.randperm(rows, generator=g).tolist()
    lo = torch.randint(-2, width + 1, (rows,), generator=g).tolist()
    hi = [a + int(torch.randint(0, width + 3, (1,), generator=g)) for a in lo]
    gq.attn_pages_free(t, r, dev(which), dev(lo), dev(hi), err=err)
    ref.pages_free(table, refs, which, lo, hi)
    same(table, t)
    same(refs, r)
    fits = ref.pages_reserve(table, refs, which, lo, hi)
    gq.attn_pages_reserve(t, r, dev(which), dev(lo), dev(hi), err=err)
    same(table, t)
    same(refs, r)
    assert int(err) == (0 if fits else gq.ATTN_ERR_PAGES)


def test_reserve_until_the_pool_is_empty():
    """More entries than one list of free pages holds, then more than there are."""
    table, refs = torch.full((3, 7000), -1, dtype=torch.int32), torch.zeros(15000, dtype=torch.int32)
    refs[5:15000:3] = 2
    t, r, err = table.to(DEV), refs.to(DEV), error()
    args = [0, 1, 2], [0, 10, 0], [5000, 4000, 3000]
    assert not ref.pages_reserve(table, refs, *args)
    gq.attn_pages_reserve(t, r, *map(dev, args), err=err)
    same(table, t)
    same(refs, r)
    assert int(err) == gq.ATTN_ERR_PAGES


def test_free_names_pages_twice_and_bad_ones():
    table = torch.tensor([[0, 1, 2, -1], [1, 99, -1, 3]], dtype=torch.int32)
    refs = torch.tensor([1, 2, 0, 1, 0], dtype=torch.int32)
    t, r, err = table.to(DEV), refs.to(DEV), error()
    # row 0 twice: an entry gives its page back once; page 99 and the free page 2 are reported
    gq.attn_pages_free(t, r, dev([0, 0, 1, 7]), dev([0, 0, 0, 0]), dev([4, 4, 4, 4]), err=err)
    same(torch.full_like(table, -1), t)
    same(torch.tensor([0, 0, 0, 0, 0], dtype=torch.int32), r)
    assert int(err) == gq.ATTN_ERR_BOUNDS


@pytest.mark.parametrize("parents,width,kids,bs,pages", [(1, 1, 1, 16, 3), (4, 20, 3, 16, 300),
                                                         (30, 1100, 2, 8, 40000),
                                                         (700, 4, 2, 5, 6000)])
def test_fork(parents, width, kids, bs, pages):
    g = gen(parents + width)
    n = parents * kids
    lens = torch.randint(0, width * bs + 1, (parents,), generator=g).tolist()
    lens[0] = width * bs if parents > 1 else 3
    table = torch.full((parents + n, width), -1, dtype=torch.int32)
    used = [-(-x // bs) for x in lens]
    table[:parents], refs = filled(g, parents, width, pages, used, share=0.1)
    if parents > 2:
        table[1, :used[1] // 2] = -1   # evicted: the fork has none either
        refs.zero_()
        for p in table[table >= 0].tolist():
            refs[p] += 1
    src = [i // kids for i in range(n)]
    dst = [parents + i for i in torch.randperm(n, generator=g).tolist()]
    cut = [max(0, lens[s] - int(torch.randint(0, 2 * bs, (1,), generator=g))) for s in src]
    t, r, err = table.to(DEV), refs.to(DEV), error()
    moves = torch.full((n + 2, 3), -7, dtype=torch.int32, device=DEV)
    count = torch.full((1,), -7, dtype=torch.int32, device=DEV)
    gq.attn_pages_fork(t, r, dev(src), dev(dst), dev(cut), bs, moves, count, err=err)
    want, ok = ref.pages_fork(table, refs, src, dst, cut, bs)
    same(table, t)
    same(refs, r)
    assert int(count) == len(want) and ok and int(err) == 0
    assert [tuple(m) for m in moves[:len(want)].tolist()] == want
    assert (moves[len(want):] == -7).all()


def test_fork_without_free_pages_and_with_bad_rows():
    table = torch.tensor([[0, 1, -1], [-1, -1, -1], [-1, -1, -1], [-1, -1, -1]], dtype=torch.int32)
    refs = torch.tensor([1, 1, 0], dtype=torch.int32)
    t, r, err = table.to(DEV), refs.to(DEV), error()
    moves, count = torch.zeros(6, 3, dtype=torch.int32, device=DEV), error()
    gq.attn_pages_fork(t, r, dev([0, 0, 0]), dev([1, 2, 3]), dev([20, 20, 16]), 16, moves, count,
                       err=err)
    want, ok = ref.pages_fork(table, refs, [0, 0, 0], [1, 2, 3], [20, 20, 16], 16)
    same(table, t)
    same(refs, r)
    assert not ok and int(err) == gq.ATTN_ERR_PAGES
    assert int(count) == 1 and moves[0].tolist() == list(want[0])
    for src, dst, n in ((9, 1, 4), (0, -1, 4), (0, 0, 4), (0, 1, -2)):
        err.zero_()
        gq.attn_pages_fork(t, r, dev([src]), dev([dst]), dev([n]), 16, moves, count, err=err)
        assert int(err) == gq.ATTN_ERR_BOUNDS and int(count) == 0
    gq.attn_pages_fork(t, r, dev([]), dev([]), dev([]), 16, moves, count)
    assert int(count) == 0


@pytest.mark.parametrize("parents,kids,free", [(3, 2, 1), (3, 2, 0), (900, 3, 2000), (900, 3, 1024),
                                               (900, 3, 1)])
def test_fork_that_runs_out_of_pages(parents, kids, free):
    """The first requests get the pages that are left, of more than one batch too;
    the moves behind *n_moves stay as they were."""
    n, bs = parents * kids, 16
    table = torch.full((parents + n, 2), -1, dtype=torch.int32)
    table[:parents, 0] = torch.randperm(parents + free, generator=gen(free))[:parents].int()
    refs = torch.zeros(parents + free, dtype=torch.int32)
    refs[table[:parents, 0].long()] = 1
    t, r, err = table.to(DEV), refs.to(DEV), error()
    src = [i // kids for i in range(n)]
    dst = [parents + i for i in range(n)]
    lens = [1 + i % 14 if i % 5 else 16 * (i % 2) for i in range(n)]  # some without a partial page
    moves = torch.full((n + 1, 3), -7, dtype=torch.int32, device=DEV)
    count = error()
    gq.attn_pages_fork(t, r, dev(src), dev(dst), dev(lens), bs, moves, count, err=err)
    want, ok = ref.pages_fork(table, refs, src, dst, lens, bs)
    same(table, t)
    same(refs, r)
    assert not ok and int(err) == gq.ATTN_ERR_PAGES and len(want) == free
    assert int(count) == free
    assert [tuple(m) for m in moves[:free].tolist()] == want
    assert (moves[free:] == -7).all()


@pytest.mark.parametrize("n,width", [(1, 2), (3, 3), (1200, 3), (3, 60000)])
def test_fork_of_rows_that_name_free_pages(n, width):
    """A free page in the source, as a full page or the partial last one, is reported and
    forked as none, also where the call itself hands that page out."""
    pages = 2 * n + 6
    table = torch.full((2 * n + 1, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    for i in range(n):         # page 2 i: in use; 2 i + 1: free, though named
        table[i, :2] = torch.tensor([2 * i, 2 * i + 1])
        refs[2 * i] = 1
    lens = [16 + 5 if i % 3 == 0 else 32 if i % 3 == 1 else 5 for i in range(n)]
    t, r, err = table.to(DEV), refs.to(DEV), error()
    moves, count = torch.full((n, 3), -7, dtype=torch.int32, device=DEV), error()
    gq.attn_pages_fork(t, r, dev(list(range(n))), dev(list(range(n, 2 * n))), dev(lens), 16, moves,
                       count, err=err)
    free = (refs == 0).nonzero()[:, 0].tolist()
    want = []
    for i in range(n):
        if i % 3 < 2:          # page 2 i shared, none behind it
            table[n + i, 0] = 2 * i
            refs[2 * i] += 1
        else:                  # five tokens of page 2 i copied
            page = free.pop(0)
            table[n + i, 0] = page
            refs[page] = 1
            want.append((2 * i, page, 5))
    same(table, t)
    same(refs, r)
    assert int(err) == gq.ATTN_ERR_BOUNDS and int(count) == len(want)
    assert [tuple(m) for m in moves[:len(want)].tolist()] == want
    assert (moves[len(want):] == -7).all()


@pytest.mark.parametrize("rows,width,pages", [(1, 1, 1), (6, 30, 400), (50, 200, 9001),
                                              (64, 3000 // 64, 70001)])
def test_compact(rows, width, pages):
    g = gen(pages)
    used = [int(torch.randint(0, width + 1, (1,), generator=g)) for _ in range(rows)]
    table, refs = filled(g, rows, width, pages, used)
    t, r, err = table.to(DEV), refs.to(DEV), error()
    want, n = ref.pages_compact(table, refs, 16)
    moves = torch.full((len(want) + 3, 3), -7, dtype=torch.int32, device=DEV)
    count, total = error(), error()
    gq.attn_pages_compact(t, r, 16, moves, count, total, err=err)
    same(table, t)
    same(refs, r)
    assert int(err) == 0 and int(count) == len(want) and int(total) == n
    assert [tuple(m) for m in moves[:len(want)].tolist()] == want
    assert (moves[len(want):] == -7).all()
    # a pool that is compact stays as it is
    gq.attn_pages_compact(t, r, 16, moves, count, total, err=err)
    same(table, t)
    assert int(count) == 0 and int(total) == n


def test_compact_with_too_little_room():
    """The first moves that fit are made; table and counts agree with them."""
    table = torch.tensor([[9, 8, 7, 1]], dtype=torch.int32)
    refs = torch.zeros(10, dtype=torch.int32)
    refs[[9, 8, 7, 1]] = 1
    t, r, err = table.to(DEV), refs.to(DEV), error()
    moves, count, total = torch.zeros(2, 3, dtype=torch.int32, device=DEV), error(), error()
    gq.attn_pages_compact(t, r, 4, moves, count, total, err=err)
    assert int(err) == gq.ATTN_ERR_WORKSPACE and int(count) == 2 and int(total) == 4
    assert moves.tolist() == [[7, 0, 4], [8, 2, 4]]
    same(torch.tensor([[9, 2, 0, 1]], dtype=torch.int32), t)
    want = torch.zeros(10, dtype=torch.int32)
    want[[9, 2, 0, 1]] = 1
    same(want, r)


@pytest.mark.parametrize("dtype,D,H,bs,layers", [
    (gq.ATTN_KV_BF16, 128, 2, 16, 1), (gq.ATTN_KV_BF16, 64, 3, 5, 40),
    (gq.ATTN_KV_FP8_E4M3, 128, 1, 24, 2), (gq.ATTN_KV_FP8_E4M3_SCALED, 64, 8, 64, 3),
    (gq.ATTN_KV_INT8_SCALED, 128, 4, 32, 2)])
@pytest.mark.parametrize("layout", [gq.ATTN_LAYOUT_BSHD, gq.ATTN_LAYOUT_BHSD])
def test_copy(dtype, D, H, bs, layers, layout):
    g = gen(D + bs)
    pages, sb = 20, 16
    scaled = dtype in (gq.ATTN_KV_FP8_E4M3_SCALED, gq.ATTN_KV_INT8_SCALED)
    wide = 2 if dtype == gq.ATTN_KV_BF16 else 1
    caches, want = [], []
    moves = [(3, 4, bs), (3, 5, bs - 1), (19, 0, 1), (2, 2, bs), (7, 8, 0), (25, 1, bs),
             (1, 9, bs + 1), (10, 11, min(bs, 17)), (6, 12, bs)]
    for _ in range(layers):
        raw = [torch.randint(0, 256, (pages, bs, H, D * wide), generator=g, dtype=torch.uint8)
               for _ in range(2)]
        scales = [torch.rand(pages * bs // sb, H, generator=g) for _ in range(2)] if scaled else []
        lay = lambda x: (x.transpose(1, 2).contiguous() if layout == gq.ATTN_LAYOUT_BHSD  # noqa: E731
                         else x.view(pages * bs, H, -1)).to(DEV)
        kv = [lay(x) for x in raw]
        if wide == 2:
            kv = [x.view(torch.bfloat16) for x in kv]
        caches.append(gq.KVCache(gq.PAGED, *kv, block_table=torch.zeros(1, 1, dtype=torch.int32,
                                                                        device=DEV),
                                 block_size=bs, dtype=dtype, layout=layout,
                                 k_scale=scales[0].to(DEV) if scaled else None,
                                 v_scale=scales[1].to(DEV) if scaled else None,
                                 scale_block=sb if scaled else 0))
        for s, d, n in moves[:8]:
            if s < pages and n <= bs:
                for x in raw:
                    x[d, :n] = x[s, :n]
                for x in scales:
                    y = x.view(pages, bs // sb, H)
                    y[d, :-(-n // sb)] = y[s, :-(-n // sb)]
        want.append((raw, scales))
    err = error()
    gq.attn_pages_copy(caches, dev(moves), dev([8]), err=err)   # the ninth is not listed
    torch.cuda.synchronize()
    assert int(err) == gq.ATTN_ERR_BOUNDS
    for c, (raw, scales) in zip(caches, want):
        for got, x in zip((c.k, c.v), raw):
            got = got.view(torch.uint8).cpu()
            got = got.transpose(1, 2) if layout == gq.ATTN_LAYOUT_BHSD else got.view(x.shape)
            assert torch.equal(got, x)
        for got, x in zip((c.k_scale, c.v_scale), scales):
            assert torch.equal(got.cpu(), x)


def test_copy_refuses_caches_of_different_shapes():
    """One launch serves all layers: heads and sizes have to agree."""
    def paged(pages, H):
        k = torch.zeros(pages * 16, H, 64, dtype=torch.bfloat16, device=DEV)
        table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
        return gq.KVCache(gq.PAGED, k, k.clone(), block_table=table, block_size=16)

    moves, count = torch.zeros(1, 3, dtype=torch.int32, device=DEV), error()
    gq.attn_pages_copy([paged(4, 2), paged(4, 2)], moves, count)
    for other in (paged(4, 1), paged(2, 2), paged(2, 4)):
        with pytest.raises(gq.AttnError):
            gq.attn_pages_copy([paged(4, 2), other], moves, count)
    gq.attn_pages_copy([], moves, count)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_serving_run(fmt):
    """Pages reserved, a prompt appended, beams forked, tokens decoded under a
    window with sinks, pages left behind freed, the pool compacted: every decode
    agrees with a cache that keeps each request's rows in one place."""
    g = gen(7)
    H, Hq, D, bs, rows, width, pages, layers = 2, 8, 128, 16, 4, 24, 60, 2
    window, sinks, n = 50, 5, 130
    dtype = {"e4m3": gq.ATTN_KV_FP8_E4M3_SCALED, "int8": gq.ATTN_KV_INT8_SCALED}[fmt]
    store = torch.uint8 if fmt == "e4m3" else torch.int8
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[0:40:3] = 1   # held by others, in no row here
    held = torch.arange(0, 40, 3, dtype=torch.int32)
    others = torch.full((1, width), -1, dtype=torch.int32)
    others[0, :len(held)] = held
    table = torch.cat([table, others.to(DEV)])

    def make(slots, **kw):
        return gq.KVCache(kw.pop("kind"),
                          *(torch.zeros(slots, H, D, dtype=store, device=DEV) for _ in range(2)),
                          dtype=dtype, scale_block=16,
                          k_scale=torch.zeros(slots // 16, H, device=DEV),
                          v_scale=torch.zeros(slots // 16, H, device=DEV), **kw)

    caches = [make(pages * bs, kind=gq.PAGED, block_table=table, block_size=bs)
              for _ in range(layers)]
    flat = [make(rows * width * bs, kind=gq.LINEAR, slots_per_seq=width * bs)
            for _ in range(layers)]
    err, moves, count, total = error(), torch.zeros(32, 3, dtype=torch.int32, device=DEV), error(), \
        error()

    def append(which, lo, hi, row_of):
        """Tokens lo .. hi - 1 of each row in `which`, in both kinds of cache."""
        t = torch.arange(lo, hi, device=DEV)
        kv = [(torch.randn(len(which) * (hi - lo), H, D, generator=g) * 2).bfloat16().to(DEV)
              for _ in range(2)]
        paged = torch.cat([table[r, t // bs].long() * bs + t % bs for r in which])
        line = torch.cat([row_of(r) * width * bs + t for r in which])
        for c, f in zip(caches, flat):
            gq.attn_kv_append(*kv, paged, c, err=err)
            gq.attn_kv_append(*kv, line, f, err=err)

    def decode(n):
        lens, pos = dev([n] * rows), dev([n - 1] * rows)
        q = torch.randn(rows, 1, Hq, D, generator=g).bfloat16().to(DEV)
        for c, f in zip(caches, flat):
            view = gq.KVCache(gq.PAGED, c.k, c.v, block_table=table[:rows], block_size=bs,
                              dtype=dtype, k_scale=c.k_scale, v_scale=c.v_scale, scale_block=16)
            a = gq.attn_decode_sinks(q, view, lens, pos, width * bs, window, sinks, 0.1, err=err)
            b = gq.attn_decode_sinks(q, f, lens, pos, width * bs, window, sinks, 0.1, err=err)
            assert torch.equal(a, b)
            assert a.any()

    gq.attn_pages_reserve(table, refs, dev([0]), dev([0]), dev([-(-n // bs)]), err=err)
    append([0], 0, n, lambda r: r)
    gq.attn_pages_fork(table, refs, dev([0, 0, 0]), dev([1, 2, 3]), dev([n] * 3), bs, moves, count,
                       err=err)
    gq.attn_pages_copy(caches, moves, count, err=err)
    assert int(count) == 3
    for f in flat:
        for x in (f.k, f.v):
            x.view(rows, width * bs, H, D)[1:] = x.view(rows, width * bs, H, D)[:1]
        for x in (f.k_scale, f.v_scale):
            x.view(rows, width * bs // 16, H)[1:] = x.view(rows, width * bs // 16, H)[:1]
    decode(n)
    every = list(range(rows))
    for step in range(40):
        gq.attn_pages_reserve(table, refs, dev(every), dev([n // bs] * rows),
                              dev([n // bs + 1] * rows), err=err)
        append(every, n, n + 1, lambda r: r)
        n += 1
        gone = max(1, (n - window) // bs)   # pages between the sinks and the window
        gq.attn_pages_free(table, refs, dev(every), dev([1] * rows), dev([gone] * rows), err=err)
        if step % 15 == 7:
            gq.attn_pages_compact(table, refs, bs, moves, count, total, err=err)
            gq.attn_pages_copy(caches, moves, count, err=err)
            assert int((refs[int(total):] != 0).sum()) == 0
        decode(n)
    assert int(err) == 0
    # every reference is a table entry
    want = torch.zeros(pages, dtype=torch.int32)
    for p in table[table >= 0].tolist():
        want[p] += 1
    same(want, refs)
    gq.attn_pages_free(table, refs, dev(every + [rows]), dev([0] * 5), dev([width] * 5), err=err)
    assert not refs.any() and int(err) == 0


def test_captured_operations():
    """A captured fork and copy follow the device's state at each replay."""
    bs, H, D, pages = 16, 1, 64, 30
    table = torch.full((3, 6), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    k, v = (torch.randn(pages * bs, H, D, device=DEV).bfloat16() for _ in range(2))
    cache = gq.KVCache(gq.PAGED, k, v, block_table=table, block_size=bs)
    src, dst, lens = dev([0, 0]), dev([1, 2]), dev([40, 40])
    zero, six = dev([0, 0]), dev([6, 6])
    moves, count, err = torch.zeros(2, 3, dtype=torch.int32, device=DEV), error(), error()
    gq.attn_pages_reserve(table, refs, dev([0]), dev([0]), dev([5]), err=err)

    def step():
        gq.attn_pages_free(table, refs, dst, zero, six, err=err)
        gq.attn_pages_fork(table, refs, src, dst, lens, bs, moves, count, err=err)
        gq.attn_pages_copy(cache, moves, count, err=err)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (33, 64, 70, 0):
        lens.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
        full, part = divmod(n, bs)
        assert int(count) == (2 if part else 0) and int(err) == 0
        for row in (1, 2):
            assert torch.equal(table[row, :full], table[0, :full])
            assert (table[row, full + (1 if part else 0):] == -1).all()
            if part:
                a, b = int(table[0, full]), int(table[row, full])
                assert a != b
                assert torch.equal(k.view(pages, bs, H, D)[a, :part], k.view(pages, bs, H, D)[b, :part])
        assert int(refs.sum()) == 5 + 2 * (full + (1 if part else 0))
