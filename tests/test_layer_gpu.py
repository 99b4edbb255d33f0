"""The decoder-layer operators on the GPU against plain 64-bit implementations.

Tolerances follow from the roundings an operator makes: a bf16 result is off by
at most 2^-8 of itself (U), an fp32 one by 2^-24 per operation; where an
operator rounds an intermediate to bf16 (attention weights before the product
with V, expert activations before the down-projection) the bound carries the
sum of the terms it enters.
"""
from __future__ import annotations

import math
import threading

import pytest
import torch

from split_bf16_gemm_swap_gb300 import gemm, layer, lowm_gemm_sync_status

pytestmark = pytest.mark.gpu

U = 2.0 ** -8                      # largest relative error of one rounding to bf16
E = 2.0 ** -24                     # of one fp32 operation
F64 = torch.float64
BF = torch.bfloat16


def rand(*shape, seed=0, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + sum(shape))
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)


def bounded(got, want, tol, what):
    assert got.shape == want.shape
    got = got.to(F64)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what + ": other elements are finite"
    off = (got - want).abs() - tol
    off = off[torch.isfinite(want)]
    assert off.numel() == 0 or off.max() <= 0, "%s: off by %.3g more than the bound" % (what, off.max())


# ------------------------------------------------------------------------------------------------ norm
def norm_reference(residual, block, post, gate, pre, scale, eps):
    r = residual.to(F64)
    size = r.abs() * abs(scale)
    if block is not None:
        y = block.to(F64)
        if post is not None:
            y = y / torch.sqrt(y.square().mean(1, keepdim=True) + eps) * post.to(F64)
        if gate is not None:
            y = y * gate.to(F64)
        r = scale * r + y
        size = size + y.abs()
    inv = 1 / torch.sqrt(r.square().mean(1, keepdim=True) + eps)
    w = pre.to(F64) if pre is not None else torch.ones_like(r[0])
    return r, r * inv * w, size, size * inv * w.abs()


def check_norm(residual, block, post, gate, pre, scale=1.0, eps=1e-6, **kw):
    r, n, r_size, n_size = norm_reference(residual, block, post, gate, pre, scale, eps)
    new, out = layer.residual_norm(residual, block, post_weight=post, gate=gate, pre_weight=pre, scale=scale, eps=eps,
                                   **kw)
    hidden = residual.shape[1]
    # Terms of r' carry a few fp32 roundings and the post norm's factor, whose
    # sum of squares has at most hidden / threads + 10 <= 42 additions.
    few = 64 * E
    rounding = few if new.dtype is torch.float32 else U
    bounded(new, r, rounding * r.abs() + few * r_size + 1e-37, "residual")
    bounded(out, n, U * n.abs() + 2 * few * n_size + 1e-37, "norm")
    assert new.shape == out.shape == (residual.shape[0], hidden)


@pytest.mark.parametrize("tokens,hidden", [(1, 1), (1, 8), (3, 7), (4, 4096), (2, 8192), (3, 8200), (2, 16384), (5, 8191),
                                           (2, 16383), (130, 2305), (257, 264), (1000, 512)])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_sizes(tokens, hidden, f32):
    res = rand(tokens, hidden, seed=1, std=3.0, dtype=torch.float32 if f32 else BF)
    block, gate = rand(tokens, hidden, seed=2), rand(tokens, hidden, seed=3)
    check_norm(res, block, rand(hidden, seed=4), gate, rand(hidden, seed=5), 0.7)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("hidden", [640, 333])
def test_norm_forms(post, gate, pre, hidden):
    t = 9
    g = {"none": None, "channel": rand(hidden, seed=3), "token": rand(t, hidden, seed=3)}[gate]
    check_norm(rand(t, hidden, seed=1), rand(t, hidden, seed=2), rand(hidden, seed=4) if post else None, g,
               rand(hidden, seed=5) if pre else None, -1.5, 1e-5)


def test_norm_without_a_block():
    res = rand(6, 1024, seed=1)
    new, out = layer.residual_norm(res, pre_weight=rand(1024, seed=2))
    assert new is res
    _, n, _, size = norm_reference(res, None, None, None, rand(1024, seed=2), 1.0, 1e-6)
    bounded(out, n, U * n.abs() + 128 * E * size, "norm")


@pytest.mark.parametrize("width,start", [(700, 0), (704, 8), (704, 3)])
def test_norm_strided_rows(width, start):
    big = rand(12, width * 2, seed=1)
    blk = rand(12, width, seed=2)
    out = torch.full((12, 999), 7.0, dtype=BF, device="cuda")
    check_norm(big[:, start:start + 600], blk[:, start:start + 600], None, rand(1, 600, seed=3)[0].expand(12, 600),
               None, out=out[:, 1:601])
    assert bool((out[:, 0] == 7).all()) and bool((out[:, 601:] == 7).all())


@pytest.mark.parametrize("hidden", [1, 5, 9, 255, 257, 2047, 4095, 8185, 8191, 16377, 16383])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_rows_off_the_16_byte_boundaries(hidden, f32):
    # contiguous rows of odd width: every row starts elsewhere; enough of them that some CTAs walk several
    tokens = 23 if hidden > 3000 else 700
    res = rand(tokens, hidden, seed=1, std=3.0, dtype=torch.float32 if f32 else BF)
    check_norm(res, rand(tokens, hidden, seed=2), rand(hidden, seed=4), rand(tokens, hidden, seed=3), rand(hidden, seed=5), 0.7)
    check_norm(res, rand(tokens, hidden, seed=2), None, rand(hidden, seed=3), None)
    # rows of a wider matrix, and tensors whose rows lie differently
    wide = rand(tokens, hidden + 8, seed=6)
    check_norm(wide[:, :hidden] if not f32 else res, wide[:, 8:], None, None, rand(hidden, seed=5))
    check_norm(res, wide[:, 3:3 + hidden], rand(hidden, seed=4), None, rand(hidden, seed=5))


def test_norm_walks_odd_rows():
    check_norm(rand(5000, 2305, seed=1), rand(5000, 2305, seed=2), rand(2305, seed=3), None, rand(2305, seed=4))
    out = torch.full((4001, 2313), 7.0, dtype=BF, device="cuda")
    res, block = rand(4001, 2313, seed=1), rand(4001, 2313, seed=2)
    check_norm(res[:, 8:], block[:, 8:], rand(2305, seed=3), None, None, out=out[:, 8:])
    assert bool((out[:, :8] == 7).all())


def test_norm_in_place():
    res, block = rand(33, 768, seed=1), rand(33, 768, seed=2)
    want = layer.residual_norm(res, block)
    new, out = layer.residual_norm(res, block, out_residual=res)
    assert new is res and torch.equal(res, want[0]) and torch.equal(out, want[1])
    want = layer.residual_norm(res, block)                     # the block's buffer takes the norm
    new, out = layer.residual_norm(res, block, out=block)
    assert out is block and torch.equal(block, want[1]) and torch.equal(new, want[0])


@pytest.mark.parametrize("hidden", [64, 98])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("swapped", [False, True])
def test_norm_outputs_side_by_side(hidden, f32, swapped):
    # both outputs' rows in the rows of one buffer
    t, size = 37, 4 if f32 else 2
    row = hidden * (size + 2)
    buf = torch.zeros(t * row, dtype=torch.uint8, device="cuda")
    at_new, at_out = (2 * hidden, 0) if swapped else (0, hidden * size)
    new = buf.view(torch.float32 if f32 else BF).as_strided((t, hidden), (row // size, 1), at_new // size)
    out = buf.view(BF).as_strided((t, hidden), (row // 2, 1), at_out // 2)
    res, block = rand(t, hidden, seed=1, dtype=torch.float32 if f32 else BF), rand(t, hidden, seed=2)
    want = layer.residual_norm(res, block)
    layer.residual_norm(res, block, out_residual=new, out=out)
    assert torch.equal(new, want[0]) and torch.equal(out, want[1])


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("tokens,hidden", [(5, 999), (4001, 1313)])
def test_norm_in_place_odd_rows(tokens, hidden, dtype):
    res, block = rand(tokens, hidden, seed=1, dtype=dtype), rand(tokens, hidden, seed=2)
    kw = dict(post_weight=rand(hidden, seed=3), gate=rand(hidden, seed=4), scale=0.5)
    want = layer.residual_norm(res, block, **kw)
    new, out = layer.residual_norm(res, block, out_residual=res, out=block, **kw)
    assert new is res and out is block and torch.equal(res, want[0]) and torch.equal(block, want[1])


@pytest.mark.parametrize("tokens,hidden", [(700, 65), (1300, 129), (3000, 385), (2500, 1313), (1100, 2305), (400, 3001),
                                           (900, 4095), (330, 8191), (330, 12001)])
@pytest.mark.parametrize("f32,gated", [(False, False), (False, True), (True, False), (True, True)])
def test_norm_odd_rows_with_and_without_edges(tokens, hidden, f32, gated):
    # widths, batches and operands on both sides of the rule that chooses between the two forms
    res = rand(tokens, hidden, seed=1, dtype=torch.float32 if f32 else BF)
    check_norm(res, rand(tokens, hidden, seed=2), rand(hidden, seed=4) if gated else None,
               rand(tokens, hidden, seed=3) if gated else None, rand(hidden, seed=5), 0.7)


def test_norm_broadcast_odd_rows():
    # one residual row for all tokens, then one block row: they lie differently from the outputs' rows
    row = rand(1, 2305, seed=1)
    check_norm(row.expand(700, -1), rand(700, 2305, seed=2), rand(2305, seed=3), None, None)
    check_norm(rand(700, 2305, seed=2), row.expand(700, -1), rand(2305, seed=3), rand(700, 2305, seed=4), None)


def test_norm_zero_rows_and_nan():
    res, block = rand(4, 512, seed=1), rand(4, 512, seed=2)
    res[1], block[1] = 0, 0
    res[2, 5] = float("nan")
    new, out = layer.residual_norm(res, block)
    assert bool((out[1] == 0).all()) and bool((new[1] == 0).all())
    assert bool(out[2].isnan().all()) and not bool(out[[0, 1, 3]].isnan().any())
    new, out = layer.residual_norm(res[:0], block[:0])
    assert out.shape == (0, 512)


# ------------------------------------------------------------------------------------------------ rope
def rope_reference(x, cos_sin, pos, sections, interleaved):
    half = cos_sin.shape[1] // 2
    pos = pos.view(-1, x.shape[0])
    y, size = x.to(F64).clone(), x.to(F64).abs()
    j = 0
    for axis, n in enumerate(sections):
        for j in range(j, j + n):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            c, s = cos_sin[pos[axis], j].to(F64)[:, None], cos_sin[pos[axis], half + j].to(F64)[:, None]
            u, v = x[..., a].to(F64), x[..., b].to(F64)
            y[..., a], y[..., b] = u * c - v * s, u * s + v * c
            size[..., a] = size[..., b] = u.abs() + v.abs()
        j += n > 0
    return y, size


def check_rope(tokens, heads, kv_heads, dim, rotary, sections, interleaved, page, shift=0, pages=None):
    width = (heads + 2 * kv_heads) * dim
    qkv = rand(tokens, width + shift, seed=1)[:, shift:]
    q, k, v = (z.unflatten(1, (-1, dim)) for z in qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
    rows = 300
    ang = torch.rand(rows, rotary // 2, device="cuda", dtype=F64) * 6.3
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    pos = torch.randint(0, rows, (len(sections), tokens), device="cuda", generator=g)
    pos = pos[0] if len(sections) == 1 else pos
    pages = pages or (2 * tokens) // page + 2
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:tokens]
    kc, vc = rand(pages, page, kv_heads, dim, seed=5), rand(pages, page, kv_heads, dim, seed=6)
    want_k, want_v = kc.to(F64).view(-1, kv_heads, dim), vc.view(-1, kv_heads, dim).clone()
    turned, size = rope_reference(k, table, pos, sections, interleaved)
    want_k[slots] = turned
    want_v[slots] = v
    size_k = torch.zeros_like(want_k)
    size_k[slots] = size
    out = layer.rope_append(q, k, v, table, pos, slots, kc, vc, sections=sections, interleaved=interleaved)
    want, size = rope_reference(q, table, pos, sections, interleaved)
    bounded(out, want, U * want.abs() + 4 * E * size + 1e-37, "q")
    bounded(kc.view(-1, kv_heads, dim), want_k, U * want_k.abs() + 4 * E * size_k + 1e-37, "k cache")
    assert torch.equal(vc.view(-1, kv_heads, dim), want_v)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv_heads,dim,rotary,sections", [
    (1, 1, 1, 128, 128, (64,)), (5, 32, 8, 128, 128, (64,)), (7, 6, 2, 128, 64, (32,)), (3, 4, 4, 64, 64, (16, 8, 8)),
    (9, 3, 1, 96, 48, (11, 13)), (4, 2, 1, 2, 2, (1,)), (6, 5, 5, 17, 10, (2, 0, 3)), (2, 2, 1, 80, 0, (0,)),
    (3, 64, 8, 256, 256, (0, 100, 28)), (2, 1, 1, 1024, 512, (256,)), (300, 8, 2, 64, 32, (4, 6, 6)), (2, 1, 1, 1, 0, (0,)),
])
def test_rope_append(tokens, heads, kv_heads, dim, rotary, sections, interleaved):
    check_rope(tokens, heads, kv_heads, dim, rotary, sections, interleaved, 16)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens", [303, 304, 400, 1216, 1300])
@pytest.mark.parametrize("heads,kv_heads,dim,rotary,sections", [
    (8, 2, 128, 128, (64,)), (7, 7, 64, 32, (5, 6, 5)), (9, 3, 96, 48, (11, 13)), (1, 1, 1024, 1024, (512,)),
    (33, 11, 48, 48, (24,)),                                                    # 16-byte pieces
    (5, 5, 17, 10, (2, 0, 3)), (5, 1, 70, 40, (20,)), (3, 1, 300, 300, (100, 50)), (11, 2, 30, 24, (12,)),   # single pairs
])
def test_rope_append_many_tokens(tokens, heads, kv_heads, dim, rotary, sections, interleaved):
    # from 2 tokens an SM on, and again from 8, a token has fewer threads with more heads each (152 SMs: 304, 1216),
    # down to one head at a time where a head alone has more pairs than that, and with a ragged last round
    check_rope(tokens, heads, kv_heads, dim, rotary, sections, interleaved, 16)


@pytest.mark.parametrize("shift", [1, 8])
def test_rope_strided(shift):
    check_rope(11, 4, 2, 64, 64, (32,), False, 7, shift=shift)


def small_rope(tokens=6):
    q, k, v = rand(tokens, 4, 64, seed=1), rand(tokens, 2, 64, seed=2), rand(tokens, 2, 64, seed=3)
    table = torch.rand(10, 64, device="cuda")
    pos = torch.arange(tokens, device="cuda")
    kc, vc = rand(3, 16, 2, 64, seed=4), rand(3, 16, 2, 64, seed=5)
    return q, k, v, table, pos, kc, vc


def test_rope_padding_and_foreign_slots():
    q, k, v, table, pos, kc, vc = small_rope()
    before = kc.clone(), vc.clone()
    slots = torch.tensor([-1, 3, 48, 1 << 40, -(1 << 40), 47], device="cuda")
    out = layer.rope_append(q, k, v, table, pos, slots, kc, vc)
    changed = (kc != before[0]).flatten(2).any(2).view(-1).nonzero()[:, 0].tolist()
    assert changed == [3, 47] and (vc != before[1]).flatten(2).any(2).view(-1).nonzero()[:, 0].tolist() == [3, 47]
    assert not bool(out.isnan().any())


def test_rope_positions_outside_the_table():
    q, k, v, table, pos, kc, vc = small_rope()
    before = kc.clone()
    pos = torch.tensor([0, -1, 10, 1 << 50, 9, 5], device="cuda")
    out = layer.rope_append(q, k, v, table, pos, torch.arange(6, device="cuda"), kc, vc)
    assert out.isnan().flatten(1).all(1).tolist() == [False, True, True, True, False, False]
    assert (kc != before).flatten(2).any(2).view(-1)[:6].tolist() == [True, False, False, False, True, True]


def test_rope_in_place_and_empty():
    q, k, v, table, pos, kc, vc = small_rope()
    slots = torch.arange(6, device="cuda")
    want = layer.rope_append(q, k, v, table, pos, slots, kc, vc)
    assert layer.rope_append(q, k, v, table, pos, slots, kc, vc, out=q) is q and torch.equal(q, want)
    assert layer.rope_append(q[:0], k[:0], v[:0], table, pos[:0], slots[:0], kc, vc).shape == (0, 4, 64)


def test_rope_head_major_cache():
    q, k, v, table, pos, _, _ = small_rope()
    kc, vc = torch.zeros(3, 2, 16, 64, dtype=BF, device="cuda"), torch.zeros(3, 2, 16, 64, dtype=BF, device="cuda")
    a, b = torch.zeros(3, 16, 2, 64, dtype=BF, device="cuda"), torch.zeros(3, 16, 2, 64, dtype=BF, device="cuda")
    slots = torch.tensor([5, 17, 40, 2, 3, 4], device="cuda")
    layer.rope_append(q, k, v, table, pos, slots, kc.transpose(1, 2), vc.transpose(1, 2))
    layer.rope_append(q, k, v, table, pos, slots, a, b)
    assert torch.equal(kc.transpose(1, 2), a) and torch.equal(vc.transpose(1, 2), b)


# ------------------------------------------------------------------------------------------- attention
def attention_reference(q, kc, vc, table, kv_lens, cu, scale, window):
    """out, the sum of weights times |v| (for the bound), lse."""
    heads, dim = q.shape[1:]
    page, kv_heads = kc.shape[1:3]
    out = torch.zeros(q.shape, dtype=F64, device="cuda")
    size = torch.zeros_like(out)
    lse = torch.full(q.shape[:2], -math.inf, dtype=F64, device="cuda")
    for b, kv in enumerate(kv_lens):
        n = cu[b + 1] - cu[b]
        kv = min(kv, table.shape[1] * page)
        if n == 0 or kv <= 0:
            continue
        at = torch.arange(kv, device="cuda")
        pages = table[b].long()[at // page]
        inside = (pages >= 0) & (pages < kc.shape[0])
        pages = pages.clamp(0, kc.shape[0] - 1)
        k = kc[pages, at % page].to(F64).masked_fill(~inside[:, None, None], 0)
        v = vc[pages, at % page].to(F64).masked_fill(~inside[:, None, None], 0)
        k, v = (z.repeat_interleave(heads // kv_heads, 1) for z in (k, v))
        pos = torch.arange(kv - n, kv, device="cuda")[:, None]
        seen = at <= pos
        if window:
            seen = seen & (at > pos - window)
        s = torch.einsum("ihd,jhd->hij", q[cu[b]:cu[b + 1]].to(F64), k) * scale
        s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True).clamp(min=-1e300)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        lse[cu[b]:cu[b + 1]] = (m + total.log())[..., 0].t()
        p = p / total.clamp(min=1e-300)
        finite = torch.where(v.isfinite(), v, 0)
        out[cu[b]:cu[b + 1]] = torch.einsum("hij,jhd->ihd", p, finite)
        size[cu[b]:cu[b + 1]] = torch.einsum("hij,jhd->ihd", p, finite.abs())
        for j in (~v.isfinite()).flatten(1).any(1).nonzero()[:, 0].tolist():     # reaches the rows that see it, no other
            for i in seen[:, j].nonzero()[:, 0].tolist():
                out[cu[b] + i] += torch.where(v[j].isfinite(), 0, p[:, i, j, None] * v[j])
    return out, size, lse


def attention_inputs(q_lens, kv_lens, heads, kv_heads, dim, page, seed=0, q_std=1.5, spare=3, garbage=float("nan")):
    per = [max(0, -(-n // page)) for n in kv_lens]
    pages = sum(per) + spare
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(q_lens), max(per + [1])), -7, dtype=torch.int32, device="cuda")
    kc, vc = rand(pages, page, kv_heads, dim, seed=seed + 1), rand(pages, page, kv_heads, dim, seed=seed + 2)
    first = 0
    for b, n in enumerate(per):
        table[b, :n] = order[first:first + n]
        if n and kv_lens[b] % page:                    # what a page holds past the sequence's end
            last = int(order[first + n - 1])
            kc[last, kv_lens[b] % page:] = garbage
            vc[last, kv_lens[b] % page:] = garbage
        first += n
    for spare_page in order[first:].tolist():
        kc[spare_page], vc[spare_page] = garbage, garbage
    cu = [sum(q_lens[:i]) for i in range(len(q_lens) + 1)]
    q = rand(cu[-1], heads, dim, seed=seed + 3, std=q_std)
    return q, kc, vc, table, cu


def check_attention(q_lens, kv_lens, heads, kv_heads, dim, page, window=0, scale=None, seed=0, q_std=1.5, **kw):
    q, kc, vc, table, cu = attention_inputs(q_lens, kv_lens, heads, kv_heads, dim, page, seed, q_std, **kw)
    run_attention(q, kc, vc, table, kv_lens, cu, window, scale)


def run_attention(q, kc, vc, table, kv_lens, cu, window=0, scale=None, **kw):
    dim = q.shape[2]
    sc = 1 / math.sqrt(dim) if scale is None else scale
    want, size, lse = attention_reference(q, kc, vc, table, kv_lens, cu, sc, window)
    got, got_lse = layer.paged_attention(q, kc, vc, table, torch.tensor(kv_lens, dtype=torch.int32, device="cuda"),
                                         torch.tensor(cu, dtype=torch.int32, device="cuda"), window=window, scale=scale,
                                         return_lse=True, **kw)
    st, detail = lowm_gemm_sync_status()
    assert st == 0, "a wait gave up: %#x" % detail
    # A score is a sum of dim products in fp32: its error, that of its
    # exponential and of the sums stay under 1e-4 for the scores drawn here
    # (|score| < 100: 100 * 2^-24 * 16 roundings); a weight is rounded to bf16
    # once before it meets V, and so is the result.
    bounded(got, want, U * want.abs() + (U + 1e-4) * size + 1e-30, "attention")
    assert torch.equal(got_lse == -math.inf, lse == -math.inf)
    seen = lse != -math.inf
    assert not bool(seen.any()) or float((got_lse.to(F64) - lse)[seen].abs().max()) <= 1e-4
    assert bool((got[~seen] == 0).all())
    return got


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (4, 4), (8, 1), (32, 8), (6, 2), (100, 1), (128, 1)])
def test_attention_heads(dim, heads, kv_heads):
    check_attention([1, 3, 1], [1, 200, 67], heads, kv_heads, dim, 16)


@pytest.mark.parametrize("kv", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4097])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_decode_lengths(kv, dim):
    check_attention([1], [kv], 8, 2, dim, 16, seed=kv)
    check_attention([1, 1, 1], [kv, 5, kv + 300], 4, 1, dim, 64, seed=kv)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_pages(page, dim):
    check_attention([1, 40, 7], [777, 300, 1030], 4, 2, dim, page, seed=page)


@pytest.mark.parametrize("q_lens,kv_lens", [
    ([128], [128]), ([129], [129]), ([64], [200]), ([33, 1, 70], [33, 900, 333]), ([300], [1000]), ([257, 2], [300, 2]),
    ([1000], [1000]), ([16] * 9, [100 * i + 16 for i in range(9)]), ([2] * 40, [i * 13 + 2 for i in range(40)]),
])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 128), (2, 2, 64), (9, 3, 64), (32, 4, 128)])
def test_attention_chunks(q_lens, kv_lens, heads, kv_heads, dim):
    check_attention(q_lens, kv_lens, heads, kv_heads, dim, 32)


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 128, 300, 5000])
def test_attention_window(window):
    check_attention([1, 50, 3], [700, 400, 90], 4, 2, 128, 16, window=window)
    check_attention([200], [900], 6, 1, 64, 64, window=window)


def test_attention_rows_that_see_nothing():
    # sequences without tokens in the cache, without new tokens, and with more new tokens than the cache holds
    check_attention([2, 0, 5, 0, 1, 3], [0, 10, 2, 0, 1, 300], 4, 2, 64, 16)
    check_attention([300, 1], [5, 0], 4, 1, 128, 16)
    q, kc, vc, table, cu = attention_inputs([2, 1], [10, 20], 4, 2, 64, 16)
    run_attention(q, kc, vc, table, [-5, 20], cu)
    run_attention(q, kc, vc, table, [0, 0], cu)


def test_attention_empty_calls():
    q, kc, vc, table, cu = attention_inputs([2], [10], 4, 2, 64, 16)
    lens, z = torch.tensor([10], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    assert layer.paged_attention(q[:0], kc, vc, table, lens, z).shape == (0, 4, 64)
    out = layer.paged_attention(q, kc, vc, table[:0], lens[:0], z[:1])           # rows of no sequence
    assert bool((out == 0).all())
    run_attention(q, kc, vc, table[:, :0], [10], cu)                             # a table without pages


def test_attention_lengths_beyond_the_table_and_foreign_pages():
    q, kc, vc, table, cu = attention_inputs([2, 3], [64, 60], 4, 2, 64, 16, garbage=0.5)
    run_attention(q, kc, vc, table, [1 << 30, 60], cu)
    table[0, 1], table[1, 0], table[1, 2] = 1 << 30, -1, kc.shape[0]
    run_attention(q, kc, vc, table, [64, 60], cu)


@pytest.mark.parametrize("q_std,scale", [(0.0, None), (30.0, 0.25), (1.0, 0.0), (4.0, -0.2)])
def test_attention_scores(q_std, scale):
    # all equal; far apart (one key takes all); no scale; negative scale
    q, kc, vc, table, cu = attention_inputs([4, 1], [500, 333], 8, 2, 128, 32, q_std=1.0)
    q = (q.float() * q_std).to(BF) if q_std < 20 else (q.float().round() * 4).to(BF)
    run_attention(q, kc, vc, table, [500, 333], cu, scale=scale)


def test_attention_infinite_scores():
    q, kc, vc, table, cu = attention_inputs([1, 2], [300, 40], 2, 1, 64, 16, garbage=0.0)
    q[0] = q[0].abs()
    page, place = int(table[0, 3]), 5
    kc[page, place] = float("-inf")                    # a score of -inf: weight 0
    run_attention(q, kc, vc, table, [300, 40], cu)


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 2, 2), (128, 8, 2), (128, 3, 1)])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("q_len,kv", [(5, 9), (20, 20), (30, 150), (100, 300), (1, 130)])
def test_attention_values_that_are_not_finite_reach_only_rows_that_see_them(dim, heads, kv_heads, window, q_len, kv):
    page = 16
    for bad in ([kv - 1], [kv - q_len // 2 - 1, kv - 2 if kv > 1 else 0], [max(0, kv - q_len - 30), kv - 1], [0],
                list(range(max(0, kv - 12), kv, 3))):
        q, kc, vc, table, cu = attention_inputs([q_len, 1], [kv, 70], heads, kv_heads, dim, page, seed=kv + q_len)
        for n, j in enumerate(bad):
            vc[int(table[0, j // page]), j % page, :, n::7] = [float("nan"), float("inf"), float("-inf")][n % 3]
        run_attention(q, kc, vc, table, [kv, 70], cu, window)


def least_time(call, n=10):
    """Shortest device time in us of `n` calls."""
    best = math.inf
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, 1e3 * a.elapsed_time(b))
    return best


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 8), (64, 16, 4)])
@pytest.mark.parametrize("window", [0, 1500])
def test_attention_values_that_are_not_finite_in_a_long_prefix(dim, heads, kv_heads, window):
    # A value that all rows of a tile see costs nothing: the products give what it gives.  One in the part that only
    # some rows see (by the chunk's own keys, or where the window ends) costs a walk over that part, at most 128 keys at
    # each end, whatever the length: 32 rows of 256 keys a warp at a few thousand cycles each are below 20 ms.
    kv, q_len, page = 4096, 64, 64
    q, kc, vc, table, cu = attention_inputs([q_len], [kv], heads, kv_heads, dim, page, seed=dim)
    lens, cu32 = torch.tensor([kv], dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")

    def call():
        return layer.paged_attention(q, kc, vc, table, lens, cu32, window=window)

    call()
    clean = least_time(call)
    first = max(0, kv - window) if window else 0                  # the last new token's first key
    where = {"common": [first + 100, kv - q_len - 200], "edges": [kv - 40, kv - 2] + ([first - 30] if window else []),
             "both": [first + 100, kv - 40]}
    for name, keys in where.items():
        kept = vc.clone()
        for n, j in enumerate(keys):
            vc[int(table[0, j // page]), j % page, :, n::5] = [float("inf"), float("nan"), float("-inf")][n % 3]
        run_attention(q, kc, vc, table, [kv], cu, window)
        took = least_time(call)
        assert took < (2 * clean + 20 if name == "common" else 20e3), (name, took, clean)
        vc.copy_(kept)


def test_attention_pages_behind_the_window_may_hold_anything():
    q, kc, vc, table, cu = attention_inputs([3, 1], [300, 200], 4, 2, 128, 16)
    clean = run_attention(q, kc, vc, table, [300, 200], cu, window=50)
    table2, kc2, vc2 = table.clone(), kc.clone(), vc.clone()
    for b, first in ((0, 300 - 3 - 50 + 1), (1, 200 - 1 - 50 + 1)):      # the first key any new token sees
        kc2[int(table[b, first // 16]), :first % 16] = float("nan")
        vc2[int(table[b, first // 16]), :first % 16] = float("inf")
        table2[b, :first // 16] = table[1 - b, 0] if b else -1
    lens, cu32 = torch.tensor([300, 200], dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    kc2[int(table[1, 0])], vc2[int(table[1, 0])] = float("nan"), float("nan")
    assert torch.equal(layer.paged_attention(q, kc2, vc2, table2, lens, cu32, window=50), clean)


@pytest.mark.parametrize("layout", ["head_major", "joined", "padded"])
def test_attention_strides(layout):
    q_lens, kv_lens, heads, kv_heads, dim, page = [3, 1, 140], [100, 301, 170], 6, 3, 64, 16
    q, kc, vc, table, cu = attention_inputs(q_lens, kv_lens, heads, kv_heads, dim, page)
    wide = torch.zeros(q.shape[0], heads * dim + 40, dtype=BF, device="cuda")
    wide[:, 3:3 + heads * dim] = q.flatten(1)
    q2 = wide[:, 3:3 + heads * dim].unflatten(1, (heads, dim))
    if layout == "head_major":
        k2, v2 = (z.transpose(1, 2).contiguous().transpose(1, 2) for z in (kc, vc))
    elif layout == "joined":
        both = torch.stack([kc, vc], 1)
        k2, v2 = both[:, 0], both[:, 1]
    else:
        both = torch.cat([kc, vc], -1)
        k2, v2 = both[..., :dim], both[..., dim:]
    wide_table = torch.zeros(table.shape[0], table.shape[1] + 5, dtype=torch.int32, device="cuda")
    wide_table[:, 2:2 + table.shape[1]] = table
    out = torch.full((q.shape[0], heads + 1, dim + 3), 9.0, dtype=BF, device="cuda")
    got = run_attention(q2, k2, v2, wide_table[:, 2:2 + table.shape[1]], kv_lens, cu, out=out[:, 1:, 1:1 + dim])
    assert bool((out[:, 0] == 9).all()) and bool((out[:, :, 0] == 9).all()) and bool((out[:, :, 1 + dim:] == 9).all())
    assert torch.equal(got, layer.paged_attention(q, kc, vc, table, torch.tensor(kv_lens, dtype=torch.int32, device="cuda"),
                                                  torch.tensor(cu, dtype=torch.int32, device="cuda")))


def test_attention_strides_of_single_dimensions():
    # a cache of one page and one head: their strides mean nothing
    page, dim = 64, 64
    q, kc, vc, table, cu = attention_inputs([2], [60], 4, 1, dim, page, spare=0)
    assert kc.shape == (1, page, 1, dim)
    kc, vc = kc.as_strided(kc.shape, (3, dim, 5, 1)), vc.as_strided(vc.shape, (0, dim, 1, 1))
    run_attention(q, kc, vc, table, [60], cu)


def test_attention_and_append_past_32_bits():
    # one buffer of 2^32 + elements serves as both caches; the sequence's pages straddle and follow 2^31 and 2^32
    kv_heads, dim, page = 2, 64, 64
    per = page * kv_heads * dim
    pages = (1 << 32) // per + 40
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs a large GPU")
    cache = torch.zeros(pages, page, kv_heads, dim, dtype=BF, device="cuda")
    ids = [5, (1 << 31) // per - 1, (1 << 31) // per + 1, (1 << 32) // per + 3, pages - 1]
    kv = [len(ids) * page - 10]
    for i in ids:
        cache[i] = rand(page, kv_heads, dim, seed=i)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    q = rand(4, 8, dim, seed=3)
    small = cache[torch.tensor(ids, device="cuda")]
    want, size, _ = attention_reference(q, small, small, torch.arange(5, dtype=torch.int32, device="cuda")[None], kv,
                                        [0, 4], 1 / 8, 0)
    got = layer.paged_attention(q, cache, cache, table, torch.tensor(kv, dtype=torch.int32, device="cuda"),
                                torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
    bounded(got, want, U * want.abs() + (U + 1e-4) * size, "attention")
    k, v = rand(2, kv_heads, dim, seed=8), rand(2, kv_heads, dim, seed=9)
    slots = torch.tensor([(pages - 1) * page + 63, ((1 << 31) // per + 1) * page], device="cuda")
    layer.rope_append(q[:2], k, v, torch.zeros(1, 0, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), slots,
                      cache, torch.zeros_like(cache[:1]).expand(pages, -1, -1, -1)[:pages])
    assert torch.equal(cache[pages - 1, 63], k[0]) and torch.equal(cache[(1 << 31) // per + 1, 0], k[1])


def test_attention_is_deterministic_and_takes_streams():
    q, kc, vc, table, cu = attention_inputs([1, 30, 1, 200], [5000, 3000, 77, 200], 16, 2, 128, 64)
    lens = torch.tensor([5000, 3000, 77, 200], dtype=torch.int32, device="cuda")
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    first = layer.paged_attention(q, kc, vc, table, lens, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(6):
        outs.append(layer.paged_attention(q, kc, vc, table, lens, cu, stream=side if i % 2 else None))
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


# ------------------------------------------------------------------------------------------------- moe
def moe_inputs(tokens, hidden, inner, experts, seed=0, exact_router=False):
    x = rand(tokens, hidden, seed=seed + 1)
    router = rand(experts, hidden, seed=seed + 2, std=1 / math.sqrt(hidden))
    if exact_router:                                   # logits are multiples of 1/4 that fp32 holds exactly: ties
        x = (x * 1.5).round().clamp(-4, 4)
        router = ((router.float() * math.sqrt(hidden)).round().clamp(-2, 2) * 0.25 / max(1, math.sqrt(hidden) // 2)).to(BF)
    w1 = rand(experts, 2 * inner, hidden, seed=seed + 3, std=1 / math.sqrt(hidden))
    w2 = rand(experts, hidden, inner, seed=seed + 4, std=1 / math.sqrt(inner))
    return x, router, w1, w2


def moe_reference(x, router, w1, w2, top_k, scoring, bias, renormalize, scale):
    x64 = x.to(F64)
    logits = x64 @ router.to(F64).t()
    p = logits.softmax(-1) if scoring == "softmax" else logits.sigmoid()
    choice = p if bias is None else p + bias.to(F64)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True)[1][:, :top_k]
    w = p.gather(1, ids) * scale
    if renormalize:
        w = w / p.gather(1, ids).sum(1, keepdim=True)
    y, var = torch.zeros_like(x64), torch.zeros_like(x64)
    inner = w2.shape[2]
    for e in ids.unique().tolist():
        rows, place = (ids == e).nonzero(as_tuple=True)
        h = x64[rows] @ w1[e].to(F64).t()
        gate, up = h[:, :inner], h[:, inner:]
        a = gate * gate.sigmoid() * up
        d = w2[e].to(F64)
        we = w[rows, place][:, None]
        y.index_add_(0, rows, (a @ d.t()) * we)
        var.index_add_(0, rows, (a.square() @ d.square().t()) * we.square())
    return y, var.sqrt()


def check_moe(tokens, hidden, inner, experts, top_k, scoring="softmax", bias=None, renormalize=True, scale=1.0, seed=0,
              exact_router=False, inputs=None, **kw):
    x, router, w1, w2 = inputs or moe_inputs(tokens, hidden, inner, experts, seed, exact_router)
    want, spread = moe_reference(x, router, w1, w2, top_k, scoring, bias, renormalize, scale)
    got = layer.moe(x, router, w1, w2, top_k, scoring=scoring, bias=bias, renormalize=renormalize, scale=scale, **kw)
    st, detail = lowm_gemm_sync_status()
    assert st == 0, "a wait gave up: %#x" % detail
    # Each activation is rounded to bf16 once (at most U of itself, errors
    # independent: 6 times the root of the sum of squares), the result once.
    bounded(got, want, U * want.abs() + 6 * U * spread + 1e-30, "moe")
    return got


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 33, 64, 100, 127, 128])
def test_moe_tokens(tokens):
    check_moe(tokens, 256, 96, 16, 3, seed=tokens)


@pytest.mark.parametrize("hidden,inner", [(8, 8), (64, 64), (72, 136), (128, 8), (8, 200), (1000, 264), (2048, 768), (520, 1032)])
def test_moe_widths(hidden, inner):
    check_moe(5, hidden, inner, 6, 2, seed=hidden)
    check_moe(40, hidden, inner, 6, 4, seed=inner)


@pytest.mark.parametrize("experts,top_k", [(1, 1), (2, 2), (3, 1), (16, 16), (64, 8), (200, 5), (1024, 16)])
def test_moe_experts(experts, top_k):
    check_moe(1, 64, 32, experts, top_k, seed=experts)
    check_moe(19, 64, 32, experts, top_k, seed=experts + 1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("use_bias", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_moe_scoring(scoring, use_bias, renormalize):
    bias = rand(24, seed=9, std=0.3, dtype=torch.float32) if use_bias else None
    check_moe(31, 128, 64, 24, 4, scoring, bias, renormalize, 2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_moe_ties_take_the_lowest_index(scoring):
    check_moe(64, 64, 32, 32, 4, scoring, exact_router=True)
    x, router, w1, w2 = moe_inputs(9, 64, 32, 12)
    check_moe(9, 64, 32, 12, 3, scoring, inputs=(x, torch.zeros_like(router), w1, w2))   # experts 0, 1, 2 for all


def test_moe_all_tokens_on_one_expert():
    x, router, w1, w2 = moe_inputs(128, 128, 96, 8)
    bias = torch.zeros(8, device="cuda")
    bias[5] = 100.0
    check_moe(128, 128, 96, 8, 1, bias=bias, inputs=(x, router, w1, w2))
    bias[2] = 50.0
    check_moe(128, 128, 96, 8, 2, "sigmoid", bias=bias, inputs=(x, router, w1, w2))


def test_moe_strided_rows():
    x, router, w1, w2 = moe_inputs(13, 64, 32, 8)
    wide = torch.zeros(13, 200, dtype=BF, device="cuda")
    wide[:, 8:72] = x
    out = torch.full((13, 131), 3.0, dtype=BF, device="cuda")
    got = check_moe(13, 64, 32, 8, 2, inputs=(wide[:, 8:72], router, w1, w2), out=out[:, 5:69])
    assert bool((out[:, :5] == 3).all()) and bool((out[:, 69:] == 3).all())
    assert torch.equal(got, layer.moe(x, router, w1, w2, 2))


def test_moe_non_finite_tokens_stay_alone():
    x, router, w1, w2 = moe_inputs(20, 64, 32, 8)
    clean = layer.moe(x, router, w1, w2, 2)
    x[3, 7], x[11, 0] = float("nan"), float("inf")
    got = layer.moe(x, router, w1, w2, 2)
    rest = [i for i in range(20) if i not in (3, 11)]
    assert torch.equal(got[rest], clean[rest]) and bool(got[3].isnan().all())
    assert layer.moe(x[:0], router, w1, w2, 2).shape == (0, 64)


def test_moe_is_deterministic_and_takes_streams():
    x, router, w1, w2 = moe_inputs(50, 512, 264, 40)
    first = layer.moe(x, router, w1, w2, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [layer.moe(x, router, w1, w2, 4, stream=side if i % 2 else None) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


# ------------------------------------------------------------------------------------------- refusals
def test_refusals():
    x, router, w1, w2 = moe_inputs(4, 64, 32, 8)
    with pytest.raises(TypeError):
        layer.moe(x.float(), router, w1, w2, 2)
    with pytest.raises(ValueError):
        layer.moe(x, router, w1[:, :, :32], w2, 2)
    with pytest.raises(ValueError):
        layer.moe(x, router, w1, w2.transpose(1, 2), 2)
    with pytest.raises(ValueError):
        layer.moe(x, router, w1, w2, 2, scoring="relu")
    with pytest.raises(layer.LowmError):
        layer.moe(x, router, w1, w2, 9)
    with pytest.raises(layer.LowmError):
        layer.moe(rand(129, 64), router, w1, w2, 2)
    q, kc, vc, table, cu = attention_inputs([2], [10], 4, 2, 64, 16)
    lens, cu = torch.tensor([10], dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        layer.paged_attention(q, kc, vc, table.long(), lens, cu)
    with pytest.raises(ValueError):
        layer.paged_attention(q, kc, vc[:-1], table, lens, cu)
    with pytest.raises(ValueError):
        layer.paged_attention(q, kc, vc, table, lens, cu[:1])
    with pytest.raises(layer.LowmError):
        layer.paged_attention(q[..., :32], kc[..., :32], vc[..., :32], table, lens, cu)
    with pytest.raises(ValueError):
        layer.paged_attention(q.cpu(), kc, vc, table, lens, cu)
    with pytest.raises(ValueError):
        layer.residual_norm(x, x[:, :32])
    with pytest.raises(ValueError):
        layer.residual_norm(x, gate=x)
    with pytest.raises(TypeError):
        layer.residual_norm(x.half(), x)
    q, k, v, table, pos, kc, vc = small_rope()
    slots = torch.arange(6, device="cuda")
    with pytest.raises(ValueError):
        layer.rope_append(q, k, v, table, pos[None].expand(3, 6), slots, kc, vc)
    with pytest.raises(ValueError):
        layer.rope_append(q, k, v, table, pos[None].expand(2, 6), slots, kc, vc, sections=(10, 10))
    with pytest.raises(TypeError):
        layer.rope_append(q, k, v, table, pos.int(), slots, kc, vc)
    with pytest.raises(ValueError):
        layer.rope_append(q, k[:, :1], v, table, pos, slots, kc, vc)


def test_graph_capture_of_a_chain():
    # the operators and the GEMM captured in one graph give what they give when launched one by one
    t, hidden, heads, kv_heads, dim = 4, 512, 8, 2, 64
    w_qkv = rand((heads + 2 * kv_heads) * dim, hidden, seed=1, std=hidden ** -0.5)
    w_o = rand(hidden, heads * dim, seed=2, std=(heads * dim) ** -0.5)
    _, router, w1, w2 = moe_inputs(t, hidden, 136, 8)
    pos, slots = torch.tensor([9, 19, 29, 39], device="cuda"), torch.tensor([9, 35, 61, 103], device="cuda")
    table = torch.tensor([[0, 9, 9], [1, 2, 9], [2, 3, 9], [4, 5, 6]], dtype=torch.int32, device="cuda")
    ang = torch.arange(64, device="cuda", dtype=F64)[:, None] * 0.1 ** torch.linspace(0, 4, dim // 2, device="cuda", dtype=F64)
    cos_sin = torch.cat([ang.cos(), ang.sin()], 1).float()
    lens, cu = (pos + 1).int(), torch.arange(5, dtype=torch.int32, device="cuda")
    kc, vc = rand(10, 16, kv_heads, dim, seed=7), rand(10, 16, kv_heads, dim, seed=8)
    x = rand(t, hidden, seed=5)

    def chain():
        _, n = layer.residual_norm(x)
        qkv = gemm(n, w_qkv)
        q, k, v = (z.unflatten(1, (-1, dim)) for z in qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
        q = layer.rope_append(q, k, v, cos_sin, pos, slots, kc, vc)
        o = layer.paged_attention(q, kc, vc, table, lens, cu)
        r, n = layer.residual_norm(x, gemm(o.flatten(1), w_o))
        return layer.residual_norm(r, layer.moe(n, router, w1, w2, 2))

    want = [z.clone() for z in chain()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain()
    for z in got:
        z.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_promised_inputs_behind_a_layer_operator():
    # A GEMM that reads A before its dependency wait (both promises) behind an operator that does not write A,
    # itself behind the kernel that does: the operator must not let the GEMM start while that kernel runs.
    from split_bf16_gemm_swap_gb300 import LOWM_FLAG_A_BEFORE_PDL_WAIT, LOWM_FLAG_W_BEFORE_PDL_WAIT
    flags = LOWM_FLAG_A_BEFORE_PDL_WAIT | LOWM_FLAG_W_BEFORE_PDL_WAIT
    hidden, n = 4096, 256
    w = rand(n, hidden, seed=1, std=hidden ** -0.5)
    small, small_out = rand(4, 512, seed=2), torch.empty(4, 512, dtype=BF, device="cuda")
    q, k, v, table, pos, kc, vc = small_rope()
    slots, rows = torch.arange(6, device="cuda"), 4096
    x, out = rand(rows, hidden, seed=3), torch.empty(rows, hidden, dtype=BF, device="cuda")
    between = {
        "norm": lambda: layer.residual_norm(small, out=small_out),
        "rope": lambda: layer.rope_append(q, k, v, table, pos, slots, kc, vc, out=q),
    }
    for name, op in between.items():
        for i in range(20):
            out.zero_()
            layer.residual_norm(x, out=out)                # long enough to be running still
            op()
            got = gemm(out[-8:], w, flags=flags)
            torch.cuda.synchronize()
            assert torch.equal(got, gemm(out[-8:], w)), (name, i)


@pytest.mark.parametrize("name", ["attention", "moe"])
def test_promised_inputs_behind_an_operator_of_two_launches(name):
    from split_bf16_gemm_swap_gb300 import LOWM_FLAG_A_BEFORE_PDL_WAIT, LOWM_FLAG_W_BEFORE_PDL_WAIT
    flags = LOWM_FLAG_A_BEFORE_PDL_WAIT | LOWM_FLAG_W_BEFORE_PDL_WAIT
    hidden, n, rows = 4096, 256, 4096
    w = rand(n, hidden, seed=1, std=hidden ** -0.5)
    x, out = rand(rows, hidden, seed=3), torch.empty(rows, hidden, dtype=BF, device="cuda")
    if name == "moe":
        small, router, w1, w2 = moe_inputs(4, 64, 32, 8)
        result = torch.empty_like(small)
        op = lambda: layer.moe(small, router, w1, w2, 2, out=result)  # noqa: E731
    else:
        q, kc, vc, table, cu = attention_inputs([1, 2], [70, 30], 4, 2, 64, 16)
        lens, cu = torch.tensor([70, 30], dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
        result = torch.empty_like(q)
        op = lambda: layer.paged_attention(q, kc, vc, table, lens, cu, out=result)  # noqa: E731
    for i in range(20):
        out.zero_()
        layer.residual_norm(x, out=out)                    # long enough to be running still
        op()
        got = gemm(out[-8:], w, flags=flags)
        torch.cuda.synchronize()
        assert torch.equal(got, gemm(out[-8:], w)), i


def test_single_token_outputs_are_checked():
    x, router, w1, w2 = moe_inputs(1, 64, 32, 8)
    small, wrong = torch.empty(1, 32, dtype=BF, device="cuda"), torch.empty(1, 64, dtype=torch.float32, device="cuda")
    for bad in (small, wrong, torch.empty(1, 64, dtype=BF)):
        with pytest.raises((ValueError, TypeError)):
            layer.moe(x, router, w1, w2, 2, out=bad)
        with pytest.raises((ValueError, TypeError)):
            layer.residual_norm(x, x, out=bad)
        with pytest.raises((ValueError, TypeError)):
            layer.residual_norm(x, x, out_residual=bad)
    with pytest.raises(ValueError):
        layer.moe(x[:, ::2], router[:, :32].contiguous(), w1[:, :, :32].contiguous(), w2[:, :32].contiguous(), 2)
    odd = torch.empty(7 * 64, dtype=BF, device="cuda").as_strided((1, 64), (3, 1))     # a single row's stride may be anything
    assert torch.equal(layer.moe(x, router, w1, w2, 2, out=odd), layer.moe(x, router, w1, w2, 2))
    new, out = layer.residual_norm(x, x, out=odd)
    assert torch.equal(out, layer.residual_norm(x, x)[1])


def test_workspaces_are_kept_for_the_default_stream_alone():
    x, router, w1, w2 = moe_inputs(4, 64, 32, 8)
    layer.release_workspaces()
    assert not layer._kept
    small = layer.moe(x, router, w1, w2, 2)
    kept = dict(layer._kept)
    assert len(kept) == 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(layer.moe(x, router, w1, w2, 2, stream=side), small) and layer._kept == kept
    q, kc, vc, table, cu = attention_inputs([1, 30], [500, 300], 16, 2, 128, 64)        # a larger one replaces it
    run_attention(q, kc, vc, table, [500, 300], cu)
    assert layer._kept[0][1].numel() > kept[0][1].numel()
    assert torch.equal(layer.moe(x, router, w1, w2, 2), small)
    layer.release_workspaces()
    assert torch.equal(layer.moe(x, router, w1, w2, 2), small)


def in_a_new_thread(call):
    """`call()`'s result from a host thread that has made no CUDA call before."""
    out = []
    t = threading.Thread(target=lambda: out.append(call()))
    t.start()
    t.join()
    assert out, "the thread's call raised"
    return out[0]


def test_first_calls_of_a_host_thread():
    # all instances and their attributes are ready, so that nothing before the tensor maps gives the thread a context
    x, router, w1, w2 = moe_inputs(4, 64, 32, 8)
    want, got = (run(lambda: layer.moe(x, router, w1, w2, 2)) for run in (lambda f: f(), in_a_new_thread))
    assert torch.equal(want, got)
    q, kc, vc, table, cu = attention_inputs([1, 3], [50, 30], 8, 2, 128, 64)
    lens, cu = torch.tensor([50, 30], dtype=torch.int32, device="cuda"), torch.tensor(cu, dtype=torch.int32, device="cuda")
    want, got = (run(lambda: layer.paged_attention(q, kc, vc, table, lens, cu)) for run in (lambda f: f(), in_a_new_thread))
    assert torch.equal(want, got)
    want = gemm(x, rand(256, 64, seed=1))
    fresh, out = rand(256, 64, seed=1), torch.empty_like(want)         # an operand whose map is not cached
    assert torch.equal(in_a_new_thread(lambda: gemm(x, fresh, out)), want)


def test_threads_on_the_default_stream():
    # every thread's calls give what they give alone: attention with many cut items, and experts, on one workspace
    def attention(seed):
        q_lens, kv_lens = [1, 30, 5], [4000 + 100 * seed, 2000, 70]
        q, kc, vc, table, cu = attention_inputs(q_lens, kv_lens, 8, 2, 128, 64, seed=seed)
        lens, cu = (torch.tensor(z, dtype=torch.int32, device="cuda") for z in (kv_lens, cu))
        return lambda: layer.paged_attention(q, kc, vc, table, lens, cu)

    def experts(seed):
        x, router, w1, w2 = moe_inputs(30 + seed, 512, 264, 40, seed=seed)
        return lambda: layer.moe(x, router, w1, w2, 4)

    calls = [attention(0), experts(1), attention(2), experts(3)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    outs = [[] for _ in calls]

    def run(i):
        for _ in range(60):
            outs[i].append(calls[i]())

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    st, detail = lowm_gemm_sync_status()
    assert st == 0, "a wait gave up: %#x" % detail
    for w, o in zip(want, outs):
        assert len(o) == 60 and all(torch.equal(w, z) for z in o)
