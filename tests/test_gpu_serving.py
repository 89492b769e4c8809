"""A prompt and the steps behind it as a serving loop makes them: norms and rotation into
a paged cache, forks of its pages, decode over the shared prefix, the cache read back."""
import pytest
import torch

import gqa_attention_kv_gb300 as gq
import kv_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt,D,R", [("bf16", 128, 1), ("bf16", 64, 3), ("int8", 128, 1),
                                     ("e4m3", 64, 2)])
def test_prompt_fork_steps_and_back(fmt, D, R):
    g = torch.Generator().manual_seed(D + R)
    B, Hq, H, bs, n, steps = 5, 8, 2, 16, 203, 4
    scaled = fmt != "bf16"
    dtype = {"bf16": gq.ATTN_KV_BF16, "int8": gq.ATTN_KV_INT8_SCALED,
             "e4m3": gq.ATTN_KV_FP8_E4M3_SCALED}[fmt]
    raw = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.uint8}[fmt]
    width = -(-(n + steps * R) // bs)
    pages = width * (B + 1) + 3
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.full((B + 1, width), -1, **i32)  # the prompt's row is the last
    refs = torch.zeros(pages, **i32)
    more = {}
    if scaled:
        more = {x: torch.zeros(pages, H, device=DEV) for x in ("k_scale", "v_scale")}
        more["scale_block"] = 16
    cache = gq.KVCache(gq.PAGED, torch.zeros(pages * bs, H, D, dtype=raw, device=DEV),
                       torch.zeros(pages * bs, H, D, dtype=raw, device=DEV), block_table=table,
                       block_size=bs, dtype=dtype, **more)
    err = torch.zeros(1, **i32)
    inv, times = gq.rope_frequencies(D, 10000.0, "yarn", 4.0, 128, device=DEV)
    turn = gq.Rope(inv, gq.ATTN_ROPE_HALF, times,
                   (1 + 0.2 * torch.randn(D, generator=g)).to(DEV),
                   (1 + 0.2 * torch.randn(D, generator=g)).to(DEV))

    def rows(count):
        fused = torch.randn(count, Hq + 2 * H, D, generator=g).bfloat16().to(DEV)
        return fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]

    def slots(row, pos):
        return table[row, pos // bs].long() * bs + pos % bs

    # the prompt: its pages, its rows
    last = torch.tensor([B], **i32)
    gq.attn_pages_reserve(table, refs, last, torch.zeros(1, **i32),
                          torch.full((1,), -(-n // bs), **i32), err=err)
    pos = torch.arange(n, **i32)
    q, k, v = rows(n)
    k_turned = torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV)
    q = gq.attn_qk_rope_append(q, k, v, pos, slots(B, pos), cache, turn, k_out=k_turned, err=err)
    if not scaled:
        got = gq.attn_prefill(q[None].contiguous(), k_turned[None], v[None].contiguous(), 0,
                              D ** -0.5)[0]
        want, mass = ref.prefill(q[None].cpu(), k_turned[None].cpu(), v[None].cpu(), 0, 0, D ** -0.5)
        ref.check_output(got, want[0], mass[0])
    # its continuations: whole pages shared, the rest copied
    kids = torch.arange(B, **i32)
    moves, count = torch.zeros(B, 3, **i32), torch.zeros(1, **i32)
    gq.attn_pages_fork(table, refs, last.expand(B).contiguous(), kids, torch.full((B,), n, **i32),
                       bs, moves, count, err=err)
    gq.attn_pages_copy(cache, moves, count, err=err)
    gq.attn_pages_reserve(table, refs, kids, torch.full((B,), n // bs, **i32),
                          torch.full((B,), width, **i32), err=err)
    prefix = torch.full((B,), n // bs * bs, **i32)
    need = gq.attn_decode_shared_workspace_size(cache, B, R, Hq, width * bs, n)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    for step in range(steps):
        lens = torch.full((B,), n + (step + 1) * R, **i32)
        pos = (lens[:, None] - R + torch.arange(R, **i32)).reshape(-1)
        row = torch.arange(B, device=DEV).repeat_interleave(R)
        q, k, v = rows(B * R)
        q = gq.attn_qk_rope_append(q, k, v, pos, slots(row, pos), cache, turn, err=err)
        out = gq.attn_decode_shared(q.view(B, R, Hq, D), cache, lens, pos, last.expand(B).contiguous(),
                                    prefix, width * bs, n, 0, D ** -0.5, workspace=ws, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    # what the cache holds, by the tables
    t = table.cpu()
    if scaled:
        kd = ref.dequantized(fmt, cache.k.cpu(), cache.k_scale.cpu(), 16)
        vd = ref.dequantized(fmt, cache.v.cpu(), cache.v_scale.cpu(), 16)
    else:
        kd, vd = cache.k.cpu().double(), cache.v.cpu().double()
    slot = lambda b, p: int(t[b, p // bs]) * bs + p % bs  # noqa: E731
    want, mass = ref.decode(q.view(B, R, Hq, D).cpu(), kd, vd, slot, lens.cpu(), pos.cpu(), 0, 0,
                            D ** -0.5)
    ref.check_output(out, want, mass, weight_bits=10)
    # attn_decode reads the same keys through the forked tables
    again = gq.attn_decode(q.view(B, R, Hq, D), cache, lens, pos, width * bs, 0, D ** -0.5)
    ref.check_output(again, want, mass)
    # one request read back as keys and values, its last row attended as a prefill does
    total = n + steps * R
    every = torch.arange(total, device=DEV)
    k_back, v_back = gq.attn_kv_read(slots(2, every), cache, err=err)
    where = [slot(2, p) for p in range(total)]
    assert ((k_back.cpu().double() - kd[where]).abs() <=
            (2.0 ** -8 + 2.0 ** -23) * kd[where].abs()).all()
    filled = torch.zeros(1, total, Hq, D, dtype=torch.bfloat16, device=DEV)
    filled[0, -1] = q.view(B, R, Hq, D)[2, -1]
    got = gq.attn_prefill(filled, k_back[None], v_back[None], 0, D ** -0.5)[0, -1]
    want, mass = ref.prefill(filled.cpu(), k_back[None].cpu(), v_back[None].cpu(), 0, 0, D ** -0.5)
    ref.check_output(got, want[0, -1], mass[0, -1])
    assert int(err) == 0
