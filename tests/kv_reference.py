"""Plain 64-bit statements of the operations on 8-bit scaled caches, windows
with sinks and pages, for the tests.  CPU tensors in, CPU tensors out."""
import math

import torch

FLOOR = 2.0 ** -64
QMAX = {"e4m3": 448.0, "int8": 127.0}


def f32(x):
    """Rounded to float32, held in 64 bits."""
    return x.float().double()


def code_values(fmt, codes):
    """The values of 8-bit codes, exactly."""
    return codes.double() if fmt == "int8" else codes.view(torch.float8_e4m3fn).double()


def encode(fmt, x, by):
    """Codes of x * by (float32 values held in 64 bits).  INT8: the exact product
    to nearest even (53 bits hold it); E4M3: the product rounded to float32, then
    to E4M3, saturating."""
    p = x * by
    if fmt == "int8":
        return torch.nan_to_num(p, nan=0.0).round().clamp(-127, 127).to(torch.int8)
    return p.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def append(fmt, codes, scale, new, slots, sb, ref=None):
    """In place, one tensor: codes [S, H, D], scale [S / sb, H], new [n, H, D]
    (bf16), slots [n].  Rows of one block are neighbours in `slots`."""
    S, H, _ = codes.shape
    x = new.double() if ref is None else f32(new.double() - ref.double())
    good = [i for i, s in enumerate(slots.tolist()) if 0 <= s < S]
    runs = []
    for i in good:
        b = int(slots[i]) // sb
        if not runs or runs[-1][0] != b:
            runs.append((b, []))
        runs[-1][1].append(i)
    for b, rows in runs:
        fresh = any(int(slots[i]) % sb == 0 for i in rows)
        for h in range(H):
            v = x[rows, h]
            a = v.abs()[torch.isfinite(v)]
            a = a.max() if a.numel() else torch.tensor(0.0, dtype=torch.float64)
            held = torch.tensor(0.0).double() if fresh else scale[b, h].double()
            now = torch.stack([held, f32(a / QMAX[fmt]),
                               torch.tensor(FLOOR, dtype=torch.float64)]).max()
            r = f32(1.0 / now)
            if held > 0 and now > held:
                blk = codes[b * sb:(b + 1) * sb, h]
                blk.copy_(encode(fmt, code_values(fmt, blk), f32(held * r)))
            scale[b, h] = now.float()
            for i in rows:
                codes[int(slots[i]), h] = encode(fmt, x[i, h], r)


def dequantized(fmt, codes, scale, sb):
    return code_values(fmt, codes) * scale.double().repeat_interleave(sb, 0)[..., None]


def ring_slot(b, t, per, sinks):
    return b * per + (t if t < sinks else sinks + (t - sinks) % (per - sinks))


def visible(t, pos, window, sinks):
    return t <= pos and (window <= 0 or pos - t < window or t < sinks)


def decode(q, k, v, slot_of, seq_lens, positions, window, sinks, scale, present=None):
    """q [B, R, Hq, D]; k, v [S, H, D] in 64 bits; slot_of(b, t) a slot, or -1 for
    a key without one.  Returns the output and, per element, sum_t p_t |v_t|
    (what relative errors of the weights act on)."""
    B, R, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    out = torch.zeros(B, R, Hq, D, dtype=torch.float64)
    mass = torch.zeros_like(out)
    for b in range(B):
        n = int(seq_lens[b])
        for r in range(R):
            pos = int(positions[b * R + r])
            ts = [t for t in range(max(0, min(n, pos + 1))) if visible(t, pos, window, sinks)]
            slots = [slot_of(b, t) for t in ts]
            slots = torch.tensor([s for s in slots if s >= 0], dtype=torch.long)
            if not len(slots):
                continue
            for h in range(H):
                s = scale * (q[b, r, h * G:(h + 1) * G].double() @ k[slots, h].T)
                p = torch.exp(s - s.max(-1, keepdim=True).values)
                p = p / p.sum(-1, keepdim=True)
                out[b, r, h * G:(h + 1) * G] = p @ v[slots, h]
                mass[b, r, h * G:(h + 1) * G] = p @ v[slots, h].abs()
    return out, mass


def prefill(q, k, v, window, sinks, scale):
    """q [B, T, Hq, D], k, v [B, T, H, D] -> output and sum p |v|, 64 bits."""
    B, T, Hq, D = q.shape
    G = Hq // k.shape[2]
    i = torch.arange(T)
    gap = i[:, None] - i[None, :]
    see = gap >= 0
    if window > 0:
        see &= (gap < window) | (i[None, :] < sinks)
    k, v = (x.double().repeat_interleave(G, 2).permute(0, 2, 1, 3) for x in (k, v))
    s = scale * (q.double().permute(0, 2, 1, 3) @ k.transpose(-1, -2))
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
    return (p @ v).permute(0, 2, 1, 3), (p @ v.abs()).permute(0, 2, 1, 3)


# Weights are rounded once: f16 (8-bit caches and prefill, half a step 2^-11) or
# two bf16 halves (bf16 caches, 2^-16 with the first half rounded and the second
# too).  2^-13 more of the mass covers scores and sums in 32 bits: a score of
# |s| <= 2^6 in log2 units carries at most 2^-17 from its own products' sums and
# 2^-18 from the float32 rounding of s - M, exp2 2^-22, and the sums over at most
# 2^13 keys grow errors of 2^-24 to at most 2^-15 as random walks of blocks.
# Last, the output's one rounding: half a bf16 step, 2^-8 of the value.
def check_output(got, ref, mass, weight_bits=11):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -weight_bits + 2.0 ** -13) * mass + 1e-30
    over = ((got - ref).abs() / bound).max().item() if ref.numel() else 0.0
    assert over <= 1.0, f"{over:.3f} of the bound"


# ------------------------------------------------------------------------ pages
def pages_free(table, refs, rows, lo, hi):
    for i, row in enumerate(rows):
        for j in range(max(0, lo[i]), min(hi[i], table.shape[1])):
            if table[row, j] >= 0:
                refs[table[row, j]] -= 1
                table[row, j] = -1


def pages_reserve(table, refs, rows, lo, hi):
    for i, row in enumerate(rows):
        for j in range(max(0, lo[i]), min(hi[i], table.shape[1])):
            if table[row, j] < 0:
                free = (refs == 0).nonzero()
                if not len(free):
                    return False
                table[row, j] = free[0, 0]
                refs[free[0, 0]] = 1
    return True


def pages_fork(table, refs, src, dst, lens, bs):
    """Returns the moves (and whether every partial page got one)."""
    moves, ok = [], True
    free = [p for p in range(len(refs)) if refs[p] == 0]
    for s, d, n in zip(src, dst, lens):
        full, part = divmod(n, bs)
        row = [-1] * table.shape[1]
        for j in range(full):
            row[j] = int(table[s, j])
            if row[j] >= 0:
                refs[row[j]] += 1
        if part and table[s, full] >= 0:
            if free:
                row[full] = free.pop(0)
                refs[row[full]] = 1
                moves.append((int(table[s, full]), row[full], part))
            else:
                ok = False
        table[d] = torch.tensor(row, dtype=torch.int32)
    return moves, ok


def pages_compact(table, refs, bs):
    used = int((refs > 0).sum())
    takes = [p for p in range(used) if refs[p] == 0]
    leaves = [p for p in range(used, len(refs)) if refs[p] > 0]
    moves = [(s, d, bs) for s, d in zip(leaves, takes)]
    for s, d, _ in moves:
        refs[d], refs[s] = refs[s].clone(), 0
        table[table == s] = d
    return moves, used
