"""Caches of 8-bit codes with a scale per block of tokens and head: append bit
for bit against the definition, decode against the values the cache holds."""
import math

import pytest
import torch

import gqa_attention_kv_gb300 as gq
import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPE = {"e4m3": gq.ATTN_KV_FP8_E4M3_SCALED, "int8": gq.ATTN_KV_INT8_SCALED}
STORE = {"e4m3": torch.uint8, "int8": torch.int8}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def to_layout(x, per, head_major):
    """[S, H, D] -> the cache tensor of a layout (blocks of `per` slots)."""
    if not head_major:
        return x.contiguous()
    return x.view(-1, per, *x.shape[1:]).transpose(1, 2).contiguous()


def from_layout(x, per, head_major):
    if not head_major:
        return x
    return x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])


class Case:
    """A cache on the CPU (slot-major) and its twin on the GPU."""

    def __init__(self, fmt, slots, H, D, sb, kind=gq.LINEAR, per=None, table=None,
                 head_major=False, k_ref=None):
        self.fmt, self.sb, self.head_major = fmt, sb, head_major
        self.per = per or slots
        self.k = torch.zeros(slots, H, D, dtype=STORE[fmt])
        self.v = torch.zeros_like(self.k)
        self.ks = torch.zeros(slots // sb, H)
        self.vs = torch.zeros_like(self.ks)
        self.k_ref, self.kind, self.table = k_ref, kind, table

    def fill(self, g):
        """Rows as an append leaves them, every block with its own size."""
        for codes, scale in ((self.k, self.ks), (self.v, self.vs)):
            S, H, D = codes.shape
            scale.copy_(torch.rand(scale.shape, generator=g) * 0.05 + 0.001)
            x = torch.randn(S, H, D, generator=g) * (36 if self.fmt == "int8" else 120)
            codes.copy_(ref.encode(self.fmt, x.double(), torch.tensor(1.0, dtype=torch.float64)))
        return self

    def cuda(self):
        args = [to_layout(x, self.per, self.head_major).to(DEV) for x in (self.k, self.v)]
        paged = self.kind == gq.PAGED
        self.gpu = gq.KVCache(
            self.kind, *args, slots_per_seq=0 if paged else self.per,
            block_table=self.table.to(DEV) if paged else None,
            block_size=self.per if paged else 0, dtype=DTYPE[self.fmt],
            layout=gq.ATTN_LAYOUT_BHSD if self.head_major else gq.ATTN_LAYOUT_BSHD,
            k_scale=self.ks.to(DEV), v_scale=self.vs.to(DEV), scale_block=self.sb,
            k_ref=None if self.k_ref is None else self.k_ref.to(DEV))
        return self.gpu

    def append(self, k_new, v_new, slots):
        ref.append(self.fmt, self.k, self.ks, k_new, slots, self.sb, self.k_ref)
        ref.append(self.fmt, self.v, self.vs, v_new, slots, self.sb)

    def check(self):
        g = self.gpu
        for mine, theirs in ((self.k, g.k), (self.v, g.v)):
            got = from_layout(theirs.cpu(), self.per, self.head_major)
            assert torch.equal(mine, got), f"{(mine != got).sum().item()} codes differ"
        assert torch.equal(self.ks, g.k_scale.cpu())
        assert torch.equal(self.vs, g.v_scale.cpu())


def new_rows(g, n, H, D, size=1.0):
    return [(torch.randn(n, H, D, generator=g) * size).bfloat16() for _ in range(2)]


def gpu_append(case, k, v, slots):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    gq.attn_kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), case.gpu, err=err)
    torch.cuda.synchronize()
    return int(err)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,H,sb,head_major", [(128, 3, 16, False), (64, 2, 32, False),
                                               (128, 2, 128, True), (64, 5, 64, True)])
def test_append_prompt_then_steps(fmt, D, H, sb, head_major):
    """A prompt that ends inside a block, then single tokens whose sizes grow and
    shrink: scales grow, the block's codes follow, a new block starts anew."""
    g = gen(D + H + sb)
    per = 3 * sb
    case = Case(fmt, 2 * per, H, D, sb, per=per, head_major=head_major)
    case.cuda()
    n = sb + sb // 2 + 1
    for size, lo, hi in [(1.0, 0, n)] + [(s, n + i, n + i + 1) for i, s in
                                         enumerate([0.5, 3.0, 20.0, 0.01, 1.0, 25.0])] + \
            [(2.0, n + 6, per)]:
        slots = torch.cat([torch.arange(lo, hi), per + torch.arange(lo, hi)])
        k, v = new_rows(g, len(slots), H, D, size)
        case.append(k, v, slots)
        assert gpu_append(case, k, v, slots) == 0
        case.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_many_rows_and_windows(fmt):
    """Enough rows for warps that look for run starts among 16: runs that begin
    and end anywhere, shuffled inside their block, and slots outside the cache."""
    g = gen(5)
    H, D, sb, blocks = 8, 128, 16, 90
    case = Case(fmt, blocks * sb, H, D, sb).fill(g)
    slots = []
    for b in torch.randperm(blocks, generator=g).tolist():
        n = int(torch.randint(1, sb + 1, (1,), generator=g))
        inside = torch.randperm(sb, generator=g)[:n] + b * sb
        slots += inside.tolist()
        if b % 7 == 0:  # in the middle of a run: its other rows still belong together
            slots[-1 - n // 2:-1 - n // 2] = [-1, blocks * sb + 5]
    slots = torch.tensor(slots)
    case.cuda()
    k, v = new_rows(g, len(slots), H, D, 3.0)
    case.append(k, v, slots)
    assert gpu_append(case, k, v, slots) == gq.ATTN_ERR_BOUNDS
    case.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_borders_of_codes(fmt):
    """Half the maximum lies on the border of two INT8 codes; zeros, the smallest
    and largest bf16 values, and a reference vector."""
    D, sb = 64, 16
    k_ref = torch.linspace(-2, 2, 2 * D).view(2, D)
    case = Case(fmt, 64, 2, D, sb, k_ref=k_ref)
    case.cuda()
    tops = torch.tensor([1 + i / 128 for i in range(128)]).bfloat16()
    k = torch.zeros(64, 2, D).bfloat16()
    k[:, 0] = tops[:64, None]
    k[:, 1] = tops[64:, None]
    k[:, :, 1:] /= 2
    k[:, :, 7:] /= 4
    v = k.clone()
    v[16:32] = 0
    v[32:48] = 2.0 ** -126
    v[48:64] *= 3e38
    slots = torch.arange(64)
    for lo in range(0, 64, 3):
        rows = slice(lo, min(64, lo + 3))
        case.append(k[rows], v[rows], slots[rows])
        assert gpu_append(case, k[rows], v[rows], slots[rows]) == 0
    case.check()


def test_append_values_that_are_not_finite():
    """Infinities saturate and leave the scale alone; a NaN stays one in E4M3 and
    is 0, reported, in INT8."""
    for fmt in ("e4m3", "int8"):
        case = Case(fmt, 32, 1, 64, 16)
        case.cuda()
        g = gen(1)
        k, v = new_rows(g, 20, 1, 64)
        k[3, 0, 5], k[4, 0, 6], k[17, 0, 7] = float("inf"), float("-inf"), float("nan")
        slots = torch.arange(20)
        case.append(k, v, slots)
        if fmt == "e4m3":  # the sign of a NaN's code is open
            assert gpu_append(case, k, v, slots) == 0
            got = case.gpu.k.cpu()
            assert (got[17, 0, 7] & 0x7F) == 0x7F
            case.k[17, 0, 7] = got[17, 0, 7]
        else:
            assert gpu_append(case, k, v, slots) == gq.ATTN_ERR_UNSUPPORTED
        case.check()
        assert torch.isfinite(case.ks).all()


def lengths(g, B, lo, hi):
    n = torch.randint(lo, hi + 1, (B,), generator=g, dtype=torch.int32)
    n[0], n[-1] = lo, hi
    return n


def decode_case(fmt, kind, B, R, Hq, H, D, lo, hi, sb, per, head_major, seed):
    g = gen(seed)
    lens = lengths(g, B, lo, hi)
    if kind == gq.PAGED:
        width = -(-hi // per)
        pages = B * width + 3
        table = torch.randperm(pages, generator=g)[:B * width].view(B, width).int()
        case = Case(fmt, pages * per, H, D, sb, kind, per, table, head_major).fill(g)
        slot = lambda b, t: int(table[b, t // per]) * per + t % per  # noqa: E731
    else:
        per = -(-hi // sb) * sb
        case = Case(fmt, B * per, H, D, sb, kind, per, None, head_major).fill(g)
        slot = lambda b, t: b * per + t  # noqa: E731
    q = torch.randn(B, R, Hq, D, generator=g).bfloat16()
    pos = (lens[:, None] - R + torch.arange(R)).reshape(-1).int()
    return case, q, lens, pos, slot


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("kind,B,R,Hq,H,D,lo,hi,sb,per,head_major,window", [
    (gq.LINEAR, 1, 1, 8, 2, 128, 1, 1, 16, 0, False, 0),        # one token
    (gq.LINEAR, 3, 1, 4, 4, 64, 1, 700, 64, 0, False, 0),       # no head sharing
    (gq.LINEAR, 2, 2, 28, 4, 128, 2, 1501, 128, 0, True, 0),    # 14 rows a KV head
    (gq.PAGED, 5, 3, 8, 2, 128, 3, 333, 16, 16, False, 0),      # 12 rows, pages of 16
    (gq.PAGED, 4, 1, 16, 2, 64, 1, 515, 16, 48, True, 0),       # pages of 48
    (gq.PAGED, 2, 7, 12, 2, 128, 7, 260, 32, 64, False, 0),     # 42 rows: three units
    (gq.PAGED, 3, 2, 8, 4, 64, 5, 400, 16, 32, False, 37),      # a window
    (gq.LINEAR, 2, 1, 10, 2, 128, 900, 1100, 32, 0, False, 129),
])
def test_decode(fmt, kind, B, R, Hq, H, D, lo, hi, sb, per, head_major, window):
    case, q, lens, pos, slot = decode_case(fmt, kind, B, R, Hq, H, D, lo, hi, sb, per, head_major,
                                           B * hi + D)
    want, mass = ref.decode(q, ref.dequantized(fmt, case.k, case.ks, sb),
                            ref.dequantized(fmt, case.v, case.vs, sb), slot, lens, pos, window, 0,
                            D ** -0.5)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = case.cuda()
    got = gq.attn_decode(q.to(DEV), cache, lens.to(DEV), pos.to(DEV), hi, window, D ** -0.5,
                         err=err)
    assert int(err) == 0
    ref.check_output(got, want, mass)
    # the answer does not depend on the run, nor on what earlier calls left behind
    ws = torch.zeros(gq.attn_decode_workspace_size(cache, B, R, Hq, hi, window),
                     dtype=torch.uint8, device=DEV)
    for _ in range(2):
        again = gq.attn_decode(q.to(DEV), cache, lens.to(DEV), pos.to(DEV), hi, window, D ** -0.5,
                               workspace=ws)
        assert torch.equal(got, again)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_scales_far_apart(fmt):
    """Blocks whose scales differ by 2^40: the weights keep their precision, and
    unwritten codes past the last token do not matter."""
    case, q, lens, pos, slot = decode_case(fmt, gq.LINEAR, 2, 1, 4, 2, 128, 100, 170, 16, 0,
                                           False, 9)
    case.vs[:3] = 2.0 ** -30
    case.vs[3:5] = 2.0 ** 10
    case.vs[13] = 3e5
    case.ks[1] = 2.0 ** -63
    want, mass = ref.decode(q, ref.dequantized(fmt, case.k, case.ks, 16),
                            ref.dequantized(fmt, case.v, case.vs, 16), slot, lens, pos, 0, 0, 0.1)
    if fmt == "e4m3":  # NaN codes where no token is
        for b in range(2):
            case.k[b * 176 + int(lens[b]):(b + 1) * 176] = 0x7F
            case.v[b * 176 + int(lens[b]):(b + 1) * 176] = 0x7F
    got = gq.attn_decode(q.to(DEV), case.cuda(), lens.to(DEV), pos.to(DEV), 170, 0, 0.1)
    ref.check_output(got, want, mass)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,R", [(64, 1), (64, 12), (128, 1), (128, 12)])
def test_decode_largest_scales(fmt, D, R):
    """Scores up to 2^20, where one key takes a row, are answered: products keep 2^-18
    of their 127 (448) sum |q|, 2^-11 of a score here, and the two largest scores lie
    further apart.  K scales from 2^103 on, whose scores pass 2^24, are reported.
    V scales of 2^126.5, whose inverse is subnormal, stand beside 2^100."""
    case, q, lens, pos, slot = decode_case(fmt, gq.LINEAR, 2, R, 4, 2, D, 300, 1500, 16, 0, False,
                                           D + R)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(answer=True):
        err.zero_()
        got = gq.attn_decode(q.to(DEV), case.cuda(), lens.to(DEV), pos.to(DEV), 1500, 0, D ** -0.5,
                             err=err)
        if answer:
            want, mass = ref.decode(q, ref.dequantized(fmt, case.k, case.ks, 16),
                                    ref.dequantized(fmt, case.v, case.vs, 16), slot, lens, pos, 0,
                                    0, D ** -0.5)
            ref.check_output(got, want, mass)
        return int(err)

    small = case.ks.clone()
    top = 13.0 if fmt == "int8" else 11.0
    for b, x in ((0, 0), (3, 1), (5, 2), (17, 4), (95, 3), (100, 4)):
        case.ks[b] = 2.0 ** (top - 4 + x) * 1.3
    assert run() == 0
    for b, x in ((0, 103), (3, 104), (5, 107), (17, 110), (95, 112), (100, 127)):
        case.ks.copy_(small)
        case.ks[b] = 2.0 ** x * 1.3
        assert run(answer=False) == gq.ATTN_ERR_UNSUPPORTED
    case.ks.copy_(small)
    one = torch.tensor(1.0, dtype=torch.float64)
    case.v.copy_(ref.encode(fmt, torch.randint(-2, 3, case.v.shape, generator=gen(1)).double(),
                            one))
    case.vs.fill_(2.0 ** 126.5)
    case.vs[::3] = 2.0 ** 100
    case.v[16:32] = 0
    assert run() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R", [1, 6])
def test_decode_queries_of_one_sign(D, R):
    """INT8 keys are multiplied as code + 128, of which 128 sum(q) is taken: sums of
    up to 255 sum |q| in 32 bits, D / 16 products and two additions of 2^-23 each,
    times what a score is multiplied with, are what the weights may be off by."""
    case, q, lens, pos, slot = decode_case("int8", gq.LINEAR, 2, R, 4, 2, D, 200, 900, 16, 0,
                                           False, D + R)
    q = (q.abs() + 2.0).bfloat16()
    q[1] = -q[1]
    case.ks.fill_(1.0 / 36)
    scale = D ** -0.5
    want, mass = ref.decode(q, ref.dequantized("int8", case.k, case.ks, 16),
                            ref.dequantized("int8", case.v, case.vs, 16), slot, lens, pos, 0, 0,
                            scale)
    off = (D / 16 + 2) * 2.0 ** -23 * 255 * q.double().abs().sum(-1).max().item() * scale / 36
    got = gq.attn_decode(q.to(DEV), case.cuda(), lens.to(DEV), pos.to(DEV), 900, 0, scale)
    got = got.double().cpu()
    # a weight and the sum of all by e^off each
    bound = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -13 + 2 * math.expm1(off)) * mass + 1e-30
    assert ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [1, 12])
def test_decode_small_weights_beside_zeros(fmt, group):
    """Key j's weight is 2^(-j / 2) of the first key's and its value stands alone in
    dim j, where all other keys have zeros: each weight shows by itself.  Weights
    down to 2^-20 of the largest keep the precision of one rounding to 11 bits."""
    n, D = 41, 128
    case = Case(fmt, 64, 1, D, 16)
    step = 0.5 * math.log(2.0)
    for j in range(n):
        case.k[j, 0, 0] = -j if fmt == "int8" else 0
        case.v[j, 0, j] = 96 if fmt == "int8" else ref.encode(
            "e4m3", torch.tensor(96.0).double(), torch.tensor(1.0).double())
    if fmt == "e4m3":  # -j as the sum of two codes
        j = torch.arange(n).double()
        for d, x in ((0, -(j // 8) * 8), (1, -(j % 8))):
            case.k[:n, 0, d] = ref.encode("e4m3", x, torch.tensor(1.0).double())
    case.ks.fill_(1.0)
    case.vs.copy_(torch.tensor([[1.0], [0.25], [3.0], [1.0]]))
    q = torch.zeros(1, 1, group, D)
    q[..., :2] = 1.0
    q = q.bfloat16()
    lens, pos = torch.tensor([n], dtype=torch.int32), torch.tensor([n - 1], dtype=torch.int32)
    want, mass = ref.decode(q, ref.dequantized(fmt, case.k, case.ks, 16),
                            ref.dequantized(fmt, case.v, case.vs, 16), lambda b, t: t, lens, pos,
                            0, 0, step)
    got = gq.attn_decode(q.to(DEV), case.cuda(), lens.to(DEV), pos.to(DEV), n, 0, step)
    ref.check_output(got, want, mass)


def test_decode_reports():
    """A page outside the pool, a length past the bound and a q past f16 are
    reported; rows without keys are zeros."""
    case, q, lens, pos, slot = decode_case("int8", gq.PAGED, 3, 1, 4, 2, 64, 20, 60, 16, 16,
                                           False, 4)
    cache = case.cuda()
    run = lambda q, lens, pos, err: gq.attn_decode(  # noqa: E731
        q.to(DEV), cache, lens.to(DEV), pos.to(DEV), 60, 0, 0.125, err=err)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = run(q, lens, pos, err)
    assert int(err) == 0
    cache.block_table[1, 0] = 10 ** 6
    bad = run(q, lens, pos, err)
    assert int(err) == gq.ATTN_ERR_BOUNDS
    assert torch.equal(bad[0], good[0]) and torch.equal(bad[2], good[2])
    skip = lambda b, t: -1 if b == 1 and t < 16 else slot(b, t)  # noqa: E731
    want, mass = ref.decode(q, ref.dequantized("int8", case.k, case.ks, 16),
                            ref.dequantized("int8", case.v, case.vs, 16), skip, lens, pos, 0, 0,
                            0.125)
    ref.check_output(bad, want, mass)
    err.zero_()
    run(q, torch.tensor([20, 61, -3], dtype=torch.int32), pos, err)
    assert int(err) == gq.ATTN_ERR_BOUNDS
    err.zero_()
    none = run(q, torch.tensor([0, 30, 60], dtype=torch.int32),
               torch.tensor([5, -1, 59], dtype=torch.int32), err)
    assert int(err) == 0 and not none[:2].any() and none[2].any()
    err.zero_()
    big = q.clone()
    big[0, 0, 0, 0] = 70000.0
    run(big, lens, pos, err)  # the bad page is in this call too: either may be the first
    assert int(err) in (gq.ATTN_ERR_UNSUPPORTED, gq.ATTN_ERR_BOUNDS)
    err.zero_()
    cache.block_table[1, 0] = case.table[1, 0]
    run(big, lens, pos, err)
    assert int(err) == gq.ATTN_ERR_UNSUPPORTED


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_fused_step_is_append_then_decode(fmt):
    case, q, lens, pos, slot = decode_case(fmt, gq.PAGED, 4, 2, 8, 2, 128, 10, 200, 16, 16, False,
                                           3)
    g = gen(8)
    k, v = new_rows(g, 8, 2, 128, 4.0)
    slots = torch.tensor([slot(b, int(lens[b]) - 2 + r) for b in range(4) for r in range(2)])
    a = case.cuda()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = gq.attn_decode_append(q.to(DEV), k.to(DEV), v.to(DEV), slots.to(DEV), a, lens.to(DEV),
                                pos.to(DEV), 200, 0, 0.1, err=err, tables_early=True)
    case.append(k, v, slots)
    case.check()
    b = case.cuda()
    want = gq.attn_decode(q.to(DEV), b, lens.to(DEV), pos.to(DEV), 200, 0, 0.1)
    assert int(err) == 0 and torch.equal(out, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,H,sb,head_major,ref_vector", [
    (128, 4, 32, False, False), (64, 5, 64, True, False), (64, 4, 128, False, True),
    (128, 4, 64, False, True), (128, 5, 128, True, False)])
def test_append_many_rows_of_long_blocks(fmt, D, H, sb, head_major, ref_vector):
    """Prompts of several requests that begin and end inside blocks whose earlier rows
    are there already, smaller and larger ones; then the same rows in disorder, with
    skipped rows among them and values that are not finite."""
    g = gen(D + H + sb)
    per = 7 * sb
    B = 9
    k_ref = torch.randn(H, D, generator=g) if ref_vector else None
    case = Case(fmt, B * per, H, D, sb, per=per, head_major=head_major, k_ref=k_ref).fill(g)
    case.cuda()
    slots = []
    for b in range(B):
        lo = int(torch.randint(0, 2 * sb, (1,), generator=g))
        hi = int(torch.randint(5 * sb, per + 1, (1,), generator=g))
        slots += range(b * per + lo, b * per + hi)
    k, v = new_rows(g, len(slots), H, D)
    grow = torch.exp(torch.randn(len(slots), 1, 1, generator=g) * 3)
    k, v = (k * grow).bfloat16(), (v * grow).bfloat16()
    at = torch.tensor(slots)
    case.append(k, v, at)
    assert gpu_append(case, k, v, at) == 0
    case.check()
    # rows of a block stay together, every third block in disorder
    order = torch.arange(len(slots))
    ends = [0] + [i for i in range(1, len(slots)) if slots[i] // sb != slots[i - 1] // sb]
    for a, b in list(zip(ends, ends[1:]))[::3]:
        order[a:b] = order[a:b][torch.randperm(b - a, generator=g)]
    at = at[order]
    at[ends[4] + 2] = -5
    at[ends[8]] = B * per + 1
    k, v = new_rows(g, len(slots), H, D, 2.0)
    v[ends[6] + 1, 0, 3], v[ends[5] + 3, 1, 2] = float("inf"), float("-inf")
    case.append(k, v, at)
    assert gpu_append(case, k, v, at) == gq.ATTN_ERR_BOUNDS
    case.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,R,per", [(128, 2, 16), (64, 2, 32), (128, 8, 16)])
def test_decode_long_shares(fmt, D, R, per):
    """64 requests that name the same pages: shares of hundreds of chunks, so every
    warp works through its tables several times over, and one request to compare with.
    Then a page outside the pool late in one of them: reported, the others unchanged."""
    B, H, Hq, L, window = 64, 8, 16, 4001, 3900
    case, q, lens, pos, slot = decode_case(fmt, gq.PAGED, 1, R, Hq, H, D, L, L, 16, per, False, D)
    want, mass = ref.decode(q, ref.dequantized(fmt, case.k, case.ks, 16),
                            ref.dequantized(fmt, case.v, case.vs, 16), slot, lens, pos, window, 0,
                            D ** -0.5)
    cache = case.cuda()
    cache.block_table = cache.block_table.repeat(B, 1).contiguous()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (q.to(DEV).repeat(B, 1, 1, 1), cache, lens.to(DEV).repeat(B), pos.to(DEV).repeat(B), L,
            window, D ** -0.5)
    got = gq.attn_decode(*args, err=err)
    assert int(err) == 0
    ref.check_output(got, want.expand(B, -1, -1, -1), mass.expand(B, -1, -1, -1))
    cache.block_table[37, (L - 200) // per] = case.k.shape[0] // per
    again = gq.attn_decode(*args, err=err)
    assert int(err) == gq.ATTN_ERR_BOUNDS
    keep = [b for b in range(B) if b != 37]
    assert torch.equal(again[keep], got[keep]) and not torch.equal(again[37], got[37])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,sb,blocks", [(128, 16, 1), (128, 16, 40), (64, 16, 40), (128, 32, 20)])
def test_append_slots_past_the_end_of_the_cache(fmt, D, sb, blocks):
    """A prompt into the last slots whose slot mapping goes on past them: the rows
    without a slot are skipped, and what lies behind the cache stays as it was."""
    H, n = 8, blocks * sb
    g = gen(D + sb + blocks)
    case = Case(fmt, n, H, D, sb).fill(g)
    cache = case.cuda()
    guarded = []
    for name in ("k", "v"):
        x = getattr(cache, name)
        big = torch.full((n + 32, H, D), 77, dtype=x.dtype, device=DEV)
        big[:n] = x
        setattr(cache, name, big[:n])
        guarded.append(big)
    at = torch.arange(n + 5)
    k, v = new_rows(g, n + 5, H, D)
    k[n:], v[n:] = 100.0, 100.0
    case.append(k, v, at)
    assert gpu_append(case, k, v, at) == gq.ATTN_ERR_BOUNDS
    case.check()
    for big in guarded:
        assert (big[n:] == 77).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,H,sb,head_major,ref_vector", [
    (128, 8, 16, False, False), (64, 8, 16, True, True), (128, 8, 64, False, True),
    (64, 5, 32, False, False)])
def test_append_short_runs(fmt, D, H, sb, head_major, ref_vector):
    """Runs of one row to seven in blocks that hold tokens, many in a warp's rows, some
    raising their block's scale, some across two warps, a few with values that are not
    finite or skipped rows beside them."""
    g = gen(D + H + sb + 1)
    blocks = 500
    k_ref = torch.randn(H, D, generator=g) if ref_vector else None
    case = Case(fmt, blocks * sb, H, D, sb, per=sb * (blocks // 4), head_major=head_major,
                k_ref=k_ref).fill(g)
    case.cuda()
    for longest in (1, 3, 7):
        at = []
        for b in torch.randperm(blocks, generator=g).tolist():
            i = int(torch.randint(0, sb, (1,), generator=g))
            m = int(torch.randint(1, longest + 1, (1,), generator=g))
            at += range(b * sb + i, min(b * sb + i + m, (b + 1) * sb))
        at = torch.tensor(at)
        at[40], at[41], at[200] = -1, blocks * sb, -7
        k, v = new_rows(g, len(at), H, D, 3.0)
        k[77, 0, 5], v[99, 1, 6] = float("inf"), float("-inf")
        case.append(k, v, at)
        assert gpu_append(case, k, v, at) == gq.ATTN_ERR_BOUNDS
        case.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("D,H,sb,head_major,ref_vector", [
    (128, 8, 16, False, False), (64, 8, 16, True, True), (128, 8, 32, False, True),
    (64, 5, 64, False, False), (128, 4, 128, True, False), (64, 1, 32, False, False)])
def test_append_long_stretches_of_skipped_rows(fmt, D, H, sb, head_major, ref_vector):
    """Padded prompts: hundreds of rows without a slot before, between and behind the
    requests' rows, and inside a block, whose rows still belong together."""
    g = gen(D + H + sb + 2)
    B, per = 5, 4 * sb
    k_ref = torch.randn(H, D, generator=g) if ref_vector else None
    case = Case(fmt, B * per, H, D, sb, per=per, head_major=head_major, k_ref=k_ref).fill(g)
    case.cuda()
    pad = lambda n: [-1] * n  # noqa: E731
    at = pad(300)
    for b in range(B):
        lo = b * per + int(torch.randint(0, 2 * sb, (1,), generator=g))
        hi = (b + 1) * per - int(torch.randint(0, sb, (1,), generator=g))
        rows = list(range(lo, hi))
        if b == 2:      # in the middle of a block
            cut = (hi - 2 * sb) // sb * sb + sb // 2 - lo
            rows[cut:cut] = pad(391)
        at += rows + pad((1, 129, 37, 260, 1000)[b])
    at = torch.tensor(at)
    at[5], at[-900] = B * per, -(2 ** 40)
    k, v = new_rows(g, len(at), H, D, 2.0)
    k[at < 0], v[at < 0] = 1e30, float("nan")
    case.append(k, v, at)
    assert gpu_append(case, k, v, at) == gq.ATTN_ERR_BOUNDS
    case.check()
    # single rows apart from each other
    slots = torch.arange(B * 4) * sb + 3
    at = torch.full((B * 4 * 50 + 700,), -1, dtype=torch.int64)
    at[333:333 + B * 4 * 50:50] = slots
    k, v = new_rows(g, len(at), H, D, 2.0)
    case.append(k, v, at)
    assert gpu_append(case, k, v, at) == gq.ATTN_ERR_BOUNDS
    case.check()


@pytest.mark.parametrize("B,H,lo,hi", [(40, 2, 1, 20000),   # one long request among short ones
                                       (1, 1, 30000, 30000)])  # one unit over the whole GPU
def test_decode_in_very_many_parts(B, H, lo, hi):
    """More parts of a unit than a warp looks up at once, added in the kernel and
    by the merge kernel."""
    g = gen(B)
    per = -(-hi // 16) * 16
    lens = torch.randint(1, 20, (B,), generator=g, dtype=torch.int32)
    lens[B // 2] = hi
    case = Case("int8", B * per, H, 64, 16, per=per)
    for codes, scale in ((case.k, case.ks), (case.v, case.vs)):
        codes.copy_(torch.randint(-127, 128, codes.shape, generator=g, dtype=torch.int8))
        scale.copy_(torch.rand(scale.shape, generator=g) * 0.02 + 0.005)
    q = torch.randn(B, 1, 2 * H, 64, generator=g).bfloat16()
    pos = lens - 1
    want, mass = ref.decode(q, ref.dequantized("int8", case.k, case.ks, 16),
                            ref.dequantized("int8", case.v, case.vs, 16),
                            lambda b, t: b * per + t, lens, pos, 0, 0, 0.125)
    got = gq.attn_decode(q.to(DEV), case.cuda(), lens.to(DEV), pos.to(DEV), hi, 0, 0.125)
    ref.check_output(got, want, mass)


@pytest.mark.parametrize("n", [100, 700, 1500, 3500])
def test_append_steps_of_many_requests(n):
    """One row a request, a warp for each or for sixteen."""
    g = gen(n)
    case = Case("e4m3", n * 16, 4, 64, 16).fill(g)
    case.cuda()
    k, v = new_rows(g, n, 4, 64, 5.0)
    slots = torch.arange(n) * 16 + torch.randint(0, 16, (n,), generator=g)
    slots = slots[torch.randperm(n, generator=g)]
    case.append(k, v, slots)
    assert gpu_append(case, k, v, slots) == 0
    case.check()


def test_one_workspace_serves_both_decodes():
    """A workspace that bf16 calls keep their zeroed counters in may serve scaled
    calls in between, graphs replayed one after the other among them."""
    g = gen(2)
    case, q, lens, pos, _ = decode_case("int8", gq.LINEAR, 2, 1, 8, 2, 128, 900, 1500, 16, 0,
                                        False, 6)
    scaled = case.cuda()
    k, v = (torch.randn(2 * case.per, 2, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    plain = gq.KVCache(gq.LINEAR, k, v, slots_per_seq=case.per)
    ws = torch.zeros(max(gq.attn_decode_workspace_size(c, 2, 1, 8, 1500) for c in (scaled, plain)),
                     dtype=torch.uint8, device=DEV)
    args = [x.to(DEV) for x in (lens, pos)]
    qd, outs = q.to(DEV), [torch.empty_like(q, device=DEV) for _ in range(2)]

    def both():
        for c, o in zip((plain, scaled), outs):
            gq.attn_decode(qd, c, *args, 1500, 0, 0.1, out=o, workspace=ws)

    both()
    first = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for _ in range(2):
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                both()
            graphs.append(gr)
        for o in outs:
            o.zero_()
        for gr in graphs * 3:
            gr.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    # the device lengths move between replays
    args[0].copy_(torch.tensor([1, 700], dtype=torch.int32))
    args[1].copy_(torch.tensor([0, 699], dtype=torch.int32))
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    moved = [o.clone() for o in outs]
    both()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(moved, outs))
