"""The 8-bit operators on the GPU against plain 64-bit implementations.

Tolerances count roundings: half a step relative to the value, 2^-8 for bf16
(U), 2^-11 for fp16 (H), 2^-24 for fp32 (E), 2^-4 for e4m3 (or 2^-10 of the scale
below its smallest normal number).
"""
from __future__ import annotations

import math
import threading

import pytest
import torch

from split_bf16_gemm_swap_gb300 import LOWM_FLAG_W_BEFORE_PDL_WAIT, fp8, layer, lowm_gemm_sync_status

pytestmark = pytest.mark.gpu

U, H, E = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
F64, BF, FP8 = torch.float64, torch.bfloat16, torch.float8_e4m3fn


def rand(*shape, seed=0, std=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + sum(shape))
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)


def codes(*shape, seed=0, std=100.0):
    return rand(*shape, seed=seed, std=std, dtype=torch.float32).clamp_(-448, 448).to(FP8)


def bounded(got, want, tol, what):
    assert got.shape == want.shape
    got = got.to(F64)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what + ": other elements are finite"
    off = ((got - want).abs() - tol)[torch.isfinite(want)]
    assert off.numel() == 0 or off.max() <= 0, "%s: off by %.3g more than the bound" % (what, off.max())


def in_order():
    status, detail = lowm_gemm_sync_status()
    assert status == 0, "status bits %#x" % detail


# ---------------------------------------------------------------------------- the format, in 64 bits
def pow2(e):
    """2 ** e exactly (the power function of 64-bit tensors on the GPU is not)."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def rounded(x):
    """Nearest e4m3 value (ties to even) of |x| <= 448."""
    f = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    step = pow2(f - 3)
    return torch.round(x / step) * step


def scale_of(amax):
    """The smallest power of two, 2^-100 at least, that brings amax to 448 or less."""
    e = torch.ceil(torch.log2(amax.to(F64).clamp(min=1e-60) / 448)).clamp(min=-100)
    e = torch.where(448 * pow2(e - 1) >= amax, e - 1, e)
    e = torch.where(448 * pow2(e) < amax, e + 1, e)
    return pow2(e.clamp(min=-100))


def quantized(x, block_rows=1):
    """Codes (their values) and scales of a matrix, from the definition."""
    rows, cols = x.shape
    x = x.to(F64)
    rb, cb = -(-rows // block_rows), -(-cols // 128)
    padded = torch.zeros(rb * block_rows, cb * 128, dtype=F64, device=x.device)
    padded[:rows, :cols] = torch.where(torch.isfinite(x), x, 0.0)
    blocks = padded.view(rb, block_rows, cb, 128)
    scale = scale_of(blocks.abs().amax((1, 3)))
    value = rounded(blocks / scale[:, None, :, None]).view(rb * block_rows, cb * 128)[:rows, :cols]
    return torch.where(torch.isfinite(x), value, math.nan), scale


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 130), (5, 128), (128, 4096), (200, 1000), (129, 257), (0, 64)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("std", [1.0, 1e-38, 1e30])
def test_quantize(rows, cols, block_rows, std):
    x = rand(rows, cols, seed=1, std=std)
    if rows > 2:
        x[1] = 0
        x[2, : cols // 2] *= 1000
    got, scale = fp8.quantize_fp8(x, block_rows)
    want, want_scale = quantized(x, block_rows)
    assert torch.equal(scale.to(F64), want_scale)
    assert torch.equal(got.to(F64), want)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_strides_and_what_is_not_finite(block_rows):
    big = rand(140, 400, seed=2)
    for start in (0, 3, 4):
        x = big[:, start:start + 260]
        x[3, 5], x[4, 200], x[5, 0:128] = math.inf, -math.inf, math.nan
        got, scale = fp8.quantize_fp8(x, block_rows)
        want, want_scale = quantized(x, block_rows)
        assert torch.equal(scale.to(F64), want_scale)
        assert torch.equal(torch.isnan(got.float()), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.to(F64)), torch.nan_to_num(want))


# --------------------------------------------------------------------------------------------- products
def check_gemm(a, sa, w, sw, c):
    m, k = a.shape
    n = w.shape[0]
    blocks = -(-k // 128)
    left = a.to(F64) * sa.to(F64).repeat_interleave(128, 1)[:, :k]
    right = w.to(F64) * sw.to(F64).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    want, size = left @ right.t(), left.abs() @ right.abs().t()
    # 128 products a block summed by the tensor cores (each addition within 2^-23 of the partial sum, truncated or not), the
    # product of the two scales, and one addition a block.
    bounded(c, want, U * want.abs() + (256 + blocks + 8) * E * size + 1e-37, "C")


SIZES = [(1, 1, 16), (4, 640, 1024), (4, 6144, 4096), (15, 63, 112), (16, 127, 144), (17, 129, 128), (32, 128, 1360), (33, 2311, 1360),
         (48, 1024, 8192), (64, 300, 4096), (65, 129, 272), (100, 4096, 2048), (127, 700, 640), (128, 6144, 4096), (128, 40, 16),
         (2, 2304, 12288), (31, 96, 8192), (7, 20000, 256), (128, 25000, 512)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm(m, n, k):
    a, sa = fp8.quantize_fp8(rand(m, k, seed=1))
    sa = sa * torch.rand(sa.shape, device="cuda").add(0.5)          # any number is a scale
    w, sw = codes(n, k, seed=2), torch.rand(-(-n // 128), -(-k // 128), device="cuda").add(0.1).mul(0.01)
    c = fp8.gemm_fp8(a, w, sw, sa)
    check_gemm(a, sa, w, sw, c)
    assert torch.equal(c, fp8.gemm_fp8(a, w, sw, sa, flags=LOWM_FLAG_W_BEFORE_PDL_WAIT, out=torch.empty_like(c)))
    in_order()


@pytest.mark.parametrize("m,n,k", SIZES)
def test_gemm_of_bf16_is_the_gemm_of_its_codes(m, n, k):
    x = rand(m, k, seed=3)
    x[0, : k // 2] = 0
    w, sw = fp8.quantize_fp8(rand(n, k, seed=4, std=0.05), 128)
    want = fp8.gemm_fp8(*fp8.quantize_fp8(x)[:1], w, sw, fp8.quantize_fp8(x)[1])
    assert torch.equal(fp8.gemm_fp8(x, w, sw), want)
    wide = rand(m, k + 24, seed=5)                                  # rows by stride, on and off 8-byte boundaries
    for start in (8, 1):
        wide[:, start:start + k] = x
        assert torch.equal(fp8.gemm_fp8(wide[:, start:start + k], w, sw), want)
    in_order()


@pytest.mark.parametrize("m", [1, 16, 29, 64, 128])
def test_gemm_of_integers_is_exact(m):
    n, k = 1000, 2048                                               # |sums| <= 2048 * 21 * 8 < 2^24, outputs rounded once
    g = torch.Generator().manual_seed(m)
    a = torch.randint(-3, 4, (m, k), generator=g).float().cuda()
    w = torch.randint(-7, 8, (n, k), generator=g).float().cuda()
    sa = 2.0 ** torch.randint(0, 2, (m, 16), generator=g).float().cuda()
    sw = 2.0 ** torch.randint(0, 2, (8, 16), generator=g).float().cuda()
    want = (a.to(F64) * sa.to(F64).repeat_interleave(128, 1)) @ (
        w.to(F64) * sw.to(F64).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)).t()
    assert torch.equal(fp8.gemm_fp8(a.to(FP8), w.to(FP8), sw, sa), want.float().to(BF))


@pytest.mark.parametrize("m,n,k", [(4, 6144, 4096), (64, 2304, 4096), (128, 6144, 2048)])
def test_gemm_repeats_its_bits(m, n, k):
    x, (w, sw) = rand(m, k, seed=1), fp8.quantize_fp8(rand(n, k, seed=2, std=0.05), 128)
    first = fp8.gemm_fp8(x, w, sw)
    for _ in range(20):
        assert torch.equal(fp8.gemm_fp8(x, w, sw), first)
    in_order()


@pytest.mark.parametrize("m", [3, 40, 128])
def test_gemm_values_that_are_not_finite_stay_in_their_row_and_column(m):
    n, k = 500, 640
    x, (w, sw) = rand(m, k, seed=1), fp8.quantize_fp8(rand(n, k, seed=2), 128)
    want = fp8.gemm_fp8(x, w, sw)
    x[1, 300] = math.inf
    w.view(torch.uint8)[77, 5] = 0x7f
    got = fp8.gemm_fp8(x, w, sw)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1], bad[:, 77] = True, True
    assert torch.equal(torch.isnan(got), bad)
    # (the infinity leaves its block's other codes as they were, unless it was the largest)
    keep = ~bad
    assert torch.equal(got[keep], want[keep])


def test_gemm_chain_reads_what_the_kernel_before_it_wrote():
    # each product's input and weights are written right before it, on the stream, without a wait
    n = 512
    x, (w, sw) = rand(8, n, seed=1), fp8.quantize_fp8(rand(n, n, seed=2, std=n ** -0.5), 128)
    weights = [fp8.quantize_fp8(rand(n, n, seed=s, std=n ** -0.5), 128)[0] for s in range(6)]
    live, y, want = torch.empty_like(w), x, x
    for v in weights:
        live.view(torch.uint8).copy_(v.view(torch.uint8))
        y = fp8.gemm_fp8(y, live, sw)
    for v in weights:
        torch.cuda.synchronize()
        want = fp8.gemm_fp8(want, v, sw)
    assert torch.equal(y, want)


# --------------------------------------------------------------------------------------------- the cache
def turned64(x, cos_sin, positions, sections, interleaved):
    half = cos_sin.shape[1] // 2
    axis = torch.repeat_interleave(torch.arange(len(sections), device=x.device), torch.tensor(sections, device=x.device))
    pos = positions.view(-1, x.shape[0])
    table = cos_sin.to(F64)
    at = pos[axis].t()                                              # [tokens, half]
    known = ((pos >= 0) & (pos < cos_sin.shape[0])).all(0)
    at = at.clamp(0, cos_sin.shape[0] - 1)
    pair = torch.arange(half, device=x.device)
    c, s = table[at, pair][:, None], table[at, half + pair][:, None]
    y = x.to(F64).clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    a, b = a.to(F64), b.to(F64)
    u, v = a * c - b * s, a * s + b * c
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = u, v
    else:
        y[..., :half], y[..., half:2 * half] = u, v
    return y, known


def append64(x, cells, scales, slots, known, block):
    """The cache after the append: code values [places, heads, dim], scales [blocks, heads], and which cells were written."""
    cells, scales = cells.to(F64).clone(), scales.to(F64).clone()
    written = torch.zeros(cells.shape[0], dtype=torch.bool, device=cells.device)
    slots = [s if k and 0 <= s < cells.shape[0] else -1 for s, k in zip(slots.tolist(), known.tolist())]
    runs = []                                                       # tokens of one block, gaps shorter than it between them
    for t, slot in enumerate(slots):
        if slot < 0:
            continue
        last = runs[-1][-1] if runs else -1
        if runs and t - last < max(block, 2) and slots[last] < slot and slots[last] // block == slot // block:
            runs[-1].append(t)
        else:
            runs.append([t])
    for run in runs:
        place, at = slots[run[0]] % block, slots[run[0]] // block
        v = x[run]
        finite = torch.where(torch.isfinite(v), v, 0.0)
        now = scale_of(finite.abs().amax((0, 2)))
        if place:
            old = slice(at * block, at * block + place)
            now = torch.maximum(now, scales[at])
            cells[old] = rounded(cells[old] * (scales[at] / now)[:, None])
        scales[at] = now
        for i, t in enumerate(run):
            value = rounded(finite[i] / now[:, None])
            cells[slots[t]] = torch.where(torch.isfinite(v[i]), value, math.nan)
            written[slots[t]] = True
    return cells, scales, written


def check_append(tokens, heads, kv_heads, dim, rotary, page, block, slots, sections=None, interleaved=False, seed=0, start=0,
                 spread=1.0, positions=None, change=None, pages=None):
    qkv = rand(tokens, (heads + 2 * kv_heads) * dim + start, seed=seed)[:, start:]
    qkv *= torch.rand(tokens, 1, device="cuda").mul(spread).exp2().to(BF)
    if change:
        change(qkv)
    q, k, v = (z.unflatten(1, (-1, dim)) for z in qkv.split([heads * dim, kv_heads * dim, kv_heads * dim], 1))
    sections = (rotary // 2,) if sections is None else sections
    cos_sin = torch.rand(300, rotary, device="cuda") * 2 - 1
    if positions is None:
        positions = torch.randint(0, 300, (len(sections), tokens), device="cuda")
        positions = positions[0].contiguous() if len(sections) == 1 else positions
    pages = (int(slots.max()) // page + 2) if pages is None else pages
    kc, vc = codes(pages, page, kv_heads, dim, seed=seed + 1), codes(pages, page, kv_heads, dim, seed=seed + 2)
    ks, vs = (2.0 ** torch.randint(-12, 1, (pages, page // block, kv_heads), device="cuda").float() for _ in range(2))
    k64, known = turned64(k, cos_sin, positions, sections, interleaved)
    q64, _ = turned64(q, cos_sin, positions, sections, interleaved)
    want_k = append64(k64, kc.view(-1, kv_heads, dim), ks.view(-1, kv_heads), slots, known, block)
    want_v = append64(v.to(F64), vc.view(-1, kv_heads, dim), vs.view(-1, kv_heads), slots, known, block)
    out = fp8.rope_append_fp8(q, k, v, cos_sin, positions, slots, kc, vc, ks, vs, sections=sections, interleaved=interleaved)
    # q: products and their sum in fp32 (terms up to |a| + |b| as |cos|, |sin| <= 1), one rounding
    size = q.to(F64).abs().amax(-1, keepdim=True)
    q64[~known] = torch.where(torch.arange(dim, device="cuda") < rotary, math.nan, q64[~known]) if (~known).any() else q64[~known]
    bounded(out, q64, U * q64.abs() + 8 * E * size, "q")
    cells, scales, _ = want_v
    assert torch.equal(vs.view(-1, kv_heads).to(F64), scales)
    got = vc.view(-1, kv_heads, dim).to(F64)
    assert torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(cells, nan=1e9))
    # k is rounded from fp32 sums: a value next to the middle of two codes may take either
    cells, scales, written = want_k
    assert torch.equal(ks.view(-1, kv_heads).to(F64), scales)
    got = kc.view(-1, kv_heads, dim).to(F64)
    assert torch.equal(torch.isnan(got), torch.isnan(cells))
    assert torch.equal(torch.nan_to_num(got[~written], nan=1e9), torch.nan_to_num(cells[~written], nan=1e9))
    off = (got - cells).abs().nan_to_num()
    step = torch.maximum(cells.abs().nan_to_num() * 2.0 ** -3, torch.tensor(2.0 ** -9, device="cuda", dtype=F64))
    assert bool((off <= step).all()) and float((off > 0).double().mean()) < 1e-4
    return kc, vc, ks, vs


def run_slots(page, lengths, pages, seed=0):
    """Slots of sequences (start, new) on shuffled pages."""
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).tolist()
    slots = []
    for start, n in lengths:
        own = [order.pop() for _ in range((start + n + page - 1) // page)]
        slots += [own[p // page] * page + p % page for p in range(start, start + n)]
    return torch.tensor(slots, device="cuda", dtype=torch.int64)


@pytest.mark.parametrize("block", [1, 8, 16, 64, 128])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (128, 64), (128, 128), (256, 128), (80, 48), (33, 10)])
def test_append(block, dim, rotary):
    page = max(block, 16)
    lengths = [(0, 37), (5, 1), (page - 1, 1), (page, 2), (30, 140), (3, 15), (0, 1)]
    slots = run_slots(page, lengths, 80)
    check_append(len(slots), 6, 2, dim, rotary, page, block, slots, seed=block + dim, spread=8.0)


@pytest.mark.parametrize("tokens", [1, 4, 33, 700])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections", [(32,), (20, 12), (8, 13, 11)])
def test_append_decode_and_axes(tokens, interleaved, sections):
    page, block = 32, 16
    slots = run_slots(page, [((7 * i) % 50, 1) for i in range(tokens)], 2 * tokens)
    check_append(tokens, 4, 4, 64, 64, page, block, slots, sections=sections, interleaved=interleaved, seed=tokens)


def test_append_strides_off_the_16_byte_boundaries():
    slots = run_slots(16, [(3, 40), (0, 9)], 8)
    for start in (1, 8):
        check_append(49, 4, 2, 128, 128, 16, 16, slots, seed=3, start=start)


def test_append_long_blocks():
    slots = run_slots(512, [(100, 700), (256, 3), (0, 600)], 8)
    for block in (256, 512):
        check_append(len(slots), 2, 2, 64, 64, 512, block, slots, seed=4, spread=6.0)


def test_append_padding_unknown_positions_and_slots_outside():
    slots = run_slots(16, [(3, 20), (0, 12)], 8)
    slots[7], slots[19], slots[25] = -1, 8 * 16 + 5, -7
    positions = torch.randint(0, 300, (32,), device="cuda")
    positions[11], positions[28] = 300, -1
    check_append(32, 4, 2, 64, 64, 16, 8, slots, seed=5, positions=positions, pages=8)


@pytest.mark.parametrize("dim", [64, 40])
def test_append_gaps(dim):
    # tokens that are not appended inside a block, before one, and for longer than a block
    page, block = 32, 16
    slots = run_slots(page, [(5, 90), (0, 40), (3, 1), (4, 50)], 16)
    for i in list(range(3, 12)) + [20, 40, 41, 60] + list(range(95, 99)) + list(range(131, 175)):
        slots[i] = -1
    check_append(len(slots), 4, 2, dim, 32, page, block, slots, seed=8, spread=8.0)


def test_append_values_that_are_not_finite():
    slots = run_slots(16, [(3, 20), (0, 12)], 8)

    def change(qkv):
        qkv[4, 4 * 64:5 * 64] = math.nan                            # a whole head of k
        qkv[9, -5], qkv[20, -64] = math.inf, -math.inf              # of v
    check_append(32, 4, 2, 64, 32, 16, 8, slots, seed=6, change=change)


def test_append_of_zeros_and_of_tiny_numbers():
    slots = run_slots(16, [(0, 16), (4, 6)], 4)
    check_append(22, 2, 2, 64, 0, 16, 16, slots, seed=7, change=lambda x: x.mul_(0))
    check_append(22, 2, 2, 64, 0, 16, 16, slots, seed=7, change=lambda x: x.mul_(1e-37))


def test_append_a_second_time_changes_nothing():
    slots = run_slots(32, [(5, 3), (0, 40)], 4)
    q, k, v = (rand(43, 2, 128, seed=s) for s in (1, 2, 3))
    table, pos = torch.rand(64, 128, device="cuda"), torch.arange(43, device="cuda")
    cache = [codes(4, 32, 2, 128, seed=4), codes(4, 32, 2, 128, seed=5), *(torch.full((4, 2, 2), 2.0 ** -9, device="cuda") for _ in range(2))]
    fp8.rope_append_fp8(q, k, v, table, pos, slots, *cache)
    before = [x.clone() for x in cache]
    fp8.rope_append_fp8(q, k, v, table, pos, slots, *cache)
    for x, y in zip(cache, before):
        assert torch.equal(x.float(), y.float())


def test_append_far_into_a_large_cache():
    pages, page, heads, dim = 70000, 256, 2, 128                    # 4.6 GB of codes: offsets pass 2^32
    kc = torch.zeros(pages, page, heads, dim, device="cuda", dtype=torch.uint8).view(FP8)
    ks = torch.ones(pages, page // 64, heads, device="cuda")
    at = (pages - 1) * page + 70
    slots = torch.arange(at, at + 20, device="cuda")
    k = rand(20, heads, dim, seed=1)
    table, pos = torch.cat([torch.ones(4, 64), torch.zeros(4, 64)], 1).cuda(), torch.zeros(20, dtype=torch.int64, device="cuda")
    fp8.rope_append_fp8(k, k, k, table, pos, slots, kc, kc, ks, ks)
    got = kc.view(-1, heads, dim)[at:at + 20].to(F64) * ks[-1, 1].to(F64)[:, None]
    assert float((got - k.to(F64)).abs().max()) <= float(k.abs().max()) * 2.0 ** -4
    q = rand(1, heads, dim, seed=2)
    page_table = torch.full((1, 1), pages - 1, device="cuda", dtype=torch.int32)
    lens, cu = torch.tensor([90], device="cuda", dtype=torch.int32), torch.tensor([0, 1], device="cuda", dtype=torch.int32)
    out = fp8.paged_attention_fp8(q, kc, kc, ks, ks, page_table, lens, cu, window=20)
    s = torch.einsum("hd,jhd->hj", q[0].to(F64), got) / math.sqrt(dim)
    want = torch.einsum("hj,jhd->hd", s.softmax(-1), got)
    assert float((out[0].to(F64) - want).abs().max()) < 0.02
    del kc
    torch.cuda.empty_cache()


# -------------------------------------------------------------------------------------------- attention
def attention64(q, kc, vc, ks, vs, table, kv_lens, cu_q, scale, window, wide):
    """out, its bound, lse; by sequence and head."""
    heads, dim = q.shape[1:]
    num_pages, page, kv_heads, _ = kc.shape
    block = page // ks.shape[1]
    out = torch.zeros(q.shape, dtype=F64, device="cuda")
    tol = torch.zeros_like(out)
    lse = torch.full(q.shape[:2], -math.inf, dtype=F64, device="cuda")
    for b in range(len(kv_lens)):
        q0, q1, kv = int(cu_q[b]), int(cu_q[b + 1]), min(int(kv_lens[b]), table.shape[1] * page)
        if q1 == q0 or kv <= 0:
            continue
        key = torch.arange(kv, device="cuda")
        pg, place = table[b, key // page].long(), key % page
        inside = (pg >= 0) & (pg < num_pages)
        pg = pg.clamp(0, num_pages - 1)

        def values(cache, scales):
            x = cache.view(torch.uint8)[pg, place].view(FP8).to(F64)
            return torch.where(inside[:, None, None], x * scales[pg, place // block].to(F64)[..., None], 0.0)

        k, v = values(kc, ks), values(vc, vs)
        at = kv - (q1 - q0) + torch.arange(q1 - q0, device="cuda")[:, None]
        seen = key <= at
        if window:
            seen &= key > at - window
        for h in range(heads):
            g = h // (heads // kv_heads)
            x = q[q0:q1, h].to(F64)
            s = scale * (x @ k[:, g].t())
            size = abs(scale) * (x.abs() @ k[:, g].abs().t())
            s = s.masked_fill(~seen, -math.inf)
            some = seen.any(1)
            p = torch.where(seen, (s - s.amax(1, keepdim=True).nan_to_num(neginf=0.0)).exp(), 0.0)
            l = p.sum(1, keepdim=True)
            w = p / l.clamp(min=1e-300)
            vh = torch.where(torch.isfinite(v[:, g]), v[:, g], 0.0)
            o = w @ vh
            poison = seen.to(F64) @ (~torch.isfinite(v[:, g])).to(F64)
            o = torch.where(poison > 0, math.nan, o)
            rows = torch.isfinite(size).all(1) | ~some
            out[q0:q1, h] = torch.where(some[:, None], o, 0.0)
            # A score is off by dim additions in fp32 and a few roundings of its size; a weight by twice that, by its own
            # rounding (fp16; with the cache widened bf16) and by the hardware's exponential.
            ds = ((dim + 16) * 2 * E * torch.where(seen, size, 0.0)).amax(1, keepdim=True).nan_to_num() + 2.0 ** -20
            weight = 2 * ds + (U if wide else H) + 16 * E
            # What a weight meets V with, w_j b_j (b_j: the scale of V), is at most 2^15 and at least 2^8 where it is the largest,
            # and fp16 numbers are 2^-24 apart below 2^-14: off by 2^-25 at most, 2^-33 of the largest, times a code.
            b_j = torch.where(inside, vs[pg, place // block, g].to(F64), 1.0)
            faint = 2.0 ** -33 * (w * b_j).amax(1, keepdim=True) * (seen.to(F64) @ (vh / b_j[:, None]).abs())
            tol[q0:q1, h] = U * out[q0:q1, h].abs().nan_to_num() + weight * (w @ vh.abs()) + faint + 1e-37
            lse[q0:q1, h] = torch.where(some, s.amax(1).nan_to_num(neginf=0.0) + l[:, 0].clamp(min=1e-300).log(), -math.inf)
    return out, tol, lse


def make_cache(kv_lens, page, block, kv_heads, dim, seed=0, width=None, spread=2.0, extra=2):
    per = [(n + page - 1) // page for n in kv_lens]
    pages = sum(per) + extra
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=g).tolist()
    width = max(max(per, default=1), 1) if width is None else width
    table = torch.zeros(len(kv_lens), width, dtype=torch.int32)
    for b, n in enumerate(per):
        for j in range(n):
            table[b, j] = order.pop()
    kc, vc = codes(pages, page, kv_heads, dim, seed=seed + 1), codes(pages, page, kv_heads, dim, seed=seed + 2)
    ks, vs = (torch.rand(pages, page // block, kv_heads, device="cuda").mul(spread).sub(8).exp2() for _ in range(2))
    return kc, vc, ks, vs, table.cuda()


def check_attention(kv_lens, q_lens, heads, kv_heads, dim, page, block, window=0, scale=None, seed=0, change=None, q=None, wide=None, **kw):
    cache = make_cache(kv_lens, page, block, kv_heads, dim, seed, **kw)
    cu = [sum(q_lens[:i]) for i in range(len(q_lens) + 1)]
    q = rand(cu[-1], heads, dim, seed=seed + 9) if q is None else q
    lens, cu_q = (torch.tensor(x, device="cuda", dtype=torch.int32) for x in (kv_lens, cu))
    if change:
        change(*cache, q)
    scale = dim ** -0.5 if scale is None else scale
    if wide is None:
        wide = widened(len(kv_lens), cu[-1], heads, kv_heads, dim, page, cache[4].shape[1])
    want, tol, lse = attention64(q, *cache, kv_lens, cu_q, scale, window, wide)
    out, got = fp8.paged_attention_fp8(q, *cache, lens, cu_q, scale=scale, window=window, return_lse=True)
    bounded(out, want, tol, "attention")
    seen = torch.isfinite(lse)
    assert torch.equal(torch.isneginf(got), ~seen)
    ok = seen & torch.isfinite(got)
    assert float((got[ok] - lse[ok]).abs().max() if ok.any() else 0) <= 1e-3
    in_order()
    return out, cache


def widened(batch, q_tokens, heads, kv_heads, dim, page, width):
    """Whether the cache is widened to bf16 first: that takes other workspace than a table without room."""
    size = lambda w: fp8.lowm_paged_attention_fp8_workspace(batch, q_tokens, heads, kv_heads, dim, page, w)   # noqa: E731
    return size(width) != size(0)


# A table with room for so many tokens makes a chunk's call worth widening; a narrow one does not.
ROOM = 60000


LENGTHS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,block", [(8, 1), (8, 8), (16, 4), (64, 16), (64, 64), (128, 32), (1024, 512)])
def test_attention_of_one_token_at_many_lengths(dim, page, block):
    check_attention(LENGTHS, [1] * len(LENGTHS), 8, 2, dim, page, block, seed=page)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (32, 8), (64, 8), (128, 1), (5, 5)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_attention_groups(heads, kv_heads, q_len):
    check_attention([700, 33, 64], [q_len] * 3, heads, kv_heads, 128, 32, 8, seed=heads)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 50, 64, 1000])
def test_attention_windows_and_drafted_tokens(dim, window):
    check_attention([300, 1000, 64, 5, 129], [7, 2, 64, 5, 1], 8, 4, dim, 16, 8, window=window, seed=window)


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 2), (64, 4, 4), (128, 4, 1)])
@pytest.mark.parametrize("window", [0, 77])
@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("room", [None, ROOM])
def test_attention_of_chunks(dim, heads, kv_heads, window, block, room):
    lens, q_lens, width = [400, 130, 700], [200, 130, 333], room and room // 32
    check_attention(lens, q_lens, heads, kv_heads, dim, 32, block, window=window, seed=dim + window, width=width, wide=bool(room))
    assert widened(3, 663, heads, kv_heads, dim, 32, width or 22) == bool(room)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,block", [(64, 64), (128, 64), (128, 128), (256, 32)])
@pytest.mark.parametrize("window,scale", [(0, None), (50, -0.2), (0, 0.0)])
def test_attention_of_chunks_with_blocks_as_long_as_a_tile(dim, page, block, window, scale):
    lens, q_lens = [400, 130, 700], [200, 130, 333]

    def change(kc, vc, ks, vs, table, q):
        vs[::2] *= 2.0 ** 20
        ks[1::3] *= -1.0
        vc.view(torch.uint8)[int(table[2, 600 // page]), 600 % page, 0, 5] = 0x7f
        vc.view(torch.uint8)[int(table[1, 0]), 3, 1, 6] = 0xff
    check_attention(lens, q_lens, 8, 2, dim, page, block, window=window, scale=scale, seed=dim + page, change=change,
                    width=ROOM // page, wide=True)
    assert widened(3, 663, 8, 2, dim, page, ROOM // page)


@pytest.mark.parametrize("block", [1, 16, 64])
def test_attention_of_chunks_of_very_different_value_scales(block):
    def change(kc, vc, ks, vs, table, q):
        vs[:, ::2] *= 2.0 ** -30
        vs[0] *= 2.0 ** 30
    check_attention([400, 130], [300, 130], 8, 2, 128, 64, block, seed=10, change=change, width=ROOM // 64, wide=True)
    assert widened(2, 430, 8, 2, 128, 64, ROOM // 64)


def test_attention_of_chunks_without_memory_to_widen():
    # a table with room for 2^27 tokens: the widened copy would pass the limit
    lens, page = [300], 64
    kc, vc, ks, vs, table = make_cache(lens, page, 16, 2, 128, seed=3)
    wide = torch.zeros(1, 1 << 21, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = rand(150, 8, 128, seed=4)
    cu = torch.tensor([0, 150], device="cuda", dtype=torch.int32)
    want, tol, _ = attention64(q, kc, vc, ks, vs, wide, lens, cu, 128 ** -0.5, 0, False)
    out = fp8.paged_attention_fp8(q, kc, vc, ks, vs, wide, torch.tensor(lens, device="cuda", dtype=torch.int32), cu)
    bounded(out, want, tol, "attention")


def test_attention_rows_that_see_nothing():
    # more new tokens than keys, no keys, no new tokens, rows behind the last sequence
    for q_lens, width in (([5, 3, 0, 2], None), ([100, 70, 0, 80], None), ([200, 170, 0, 180], ROOM // 16)):
        lens = [2, 0, 40, 60]
        kc, vc, ks, vs, table = make_cache(lens, 16, 8, 2, 64, seed=1, width=width)
        assert widened(4, sum(q_lens) + 3, 4, 2, 64, 16, table.shape[1]) == bool(width)
        cu = [sum(q_lens[:i]) for i in range(5)]
        q = rand(cu[-1] + 3, 4, 64, seed=2)
        cu_q = torch.tensor(cu, device="cuda", dtype=torch.int32)
        want, tol, lse = attention64(q, kc, vc, ks, vs, table, lens, cu_q, 0.125, 0, bool(width))
        out, got = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, torch.tensor(lens, device="cuda", dtype=torch.int32), cu_q,
                                           scale=0.125, return_lse=True)
        bounded(out, want, tol, "attention")
        assert torch.equal(torch.isneginf(got), torch.isneginf(lse))
        assert bool((out[cu[-1]:] == 0).all())


def test_attention_of_an_empty_batch():
    kc, vc, ks, vs, table = make_cache([5], 16, 8, 2, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = fp8.paged_attention_fp8(rand(3, 4, 64), kc, vc, ks, vs, table[:0], none, cu)
    assert bool((out == 0).all())
    assert fp8.paged_attention_fp8(rand(0, 4, 64), kc, vc, ks, vs, table[:0], none, cu).shape == (0, 4, 64)


@pytest.mark.parametrize("q_lens,width", [([1, 1, 1], None), ([9, 5, 7], None), ([100, 90, 70], None), ([100, 90, 70], ROOM // 64)])
def test_attention_what_no_row_sees_may_hold_anything(q_lens, width):
    lens, page, block = [100, 130, 71], 64, 16

    def change(kc, vc, ks, vs, table, q):
        for b, n in enumerate(lens):
            last = int(table[b, (n - 1) // page])
            for c in (kc, vc):
                c.view(torch.uint8)[last, (n - 1) % page + 1:] = 0x7f
            first_free = -(-((n - 1) % page + 1) // block)
            for s in (ks, vs):
                s[last, first_free:] = math.nan
        free = [i for i in range(kc.shape[0]) if i not in table.flatten().tolist()]
        for c in (kc, vc):
            c.view(torch.uint8)[free] = 0xff
    check_attention(lens, q_lens, 4, 2, 128, page, block, seed=5, change=change, width=width)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,width", [([1, 1], None), ([6, 20], None), ([120, 80], None), ([120, 80], ROOM // 32)])
@pytest.mark.parametrize("window", [0, 30])
def test_attention_nan_codes_reach_the_rows_that_see_them(dim, q_lens, window, width):
    lens, page = [200, 150], 32

    def change(kc, vc, ks, vs, table, q):
        for b, n in enumerate(lens):
            for key, d in ((n - 3, 5), (n - 15, 6), (n - q_lens[b], 7), (n - 40, 8), (2, 9)):
                vc.view(torch.uint8)[int(table[b, key // page]), key % page, 0, d] = 0xff
    out, _ = check_attention(lens, q_lens, 4, 2, dim, page, 8, window=window, seed=6, change=change, width=width)
    assert torch.isnan(out).any() and not torch.isnan(out).all()


def test_attention_nan_keys_and_queries():
    lens, q_lens = [200, 150], [6, 3]
    kc, vc, ks, vs, table = make_cache(lens, 32, 8, 2, 64, seed=7)
    kc.view(torch.uint8)[int(table[0, 197 // 32]), 197 % 32, 1, 3] = 0x7f      # seen by tokens 3.. of sequence 0
    q = rand(9, 4, 64, seed=8)
    q[7, 2, 10], q[8, 0, 1] = math.inf, math.nan
    cu = torch.tensor([0, 6, 9], device="cuda", dtype=torch.int32)
    out = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, torch.tensor(lens, device="cuda", dtype=torch.int32), cu)
    bad = torch.isnan(out).any(-1)
    want = torch.zeros_like(bad)
    want[3:6, 2:] = True
    want[7, 2], want[8, 0] = True, True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(out).all(-1), want)


def test_attention_pages_outside_the_cache_read_as_zeros():
    def change(kc, vc, ks, vs, table, q):
        table[0, 1], table[1, 0] = -1, kc.shape[0]
    for q_lens, width in (([1, 2], None), ([80, 70], None), ([120, 110], ROOM // 32)):
        check_attention([150, 120], q_lens, 4, 2, 64, 32, 16, seed=8, change=change, width=width)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
@pytest.mark.parametrize("q_lens,width", [([1, 4], None), ([190, 90], None), ([190, 90], ROOM // 16)])
def test_attention_scales_of_scores(scale, q_lens, width):
    check_attention([300, 100], q_lens, 4, 2, 64, 16, 8, scale=scale, seed=9, width=width)


@pytest.mark.parametrize("block", [1, 16])
def test_attention_of_very_different_value_scales(block):
    # neighbouring blocks whose scales are 2^30 apart: the small ones' weights keep their digits
    def change(kc, vc, ks, vs, table, q):
        vs[:, ::2] *= 2.0 ** -30
    check_attention([500, 64], [1, 2], 4, 2, 128, 32, block, seed=10, change=change)


def test_attention_of_a_sink_and_many_faint_keys():
    # one key takes nearly everything; of the others each has a weight around 2^-23, together about a hundredth
    n, page, dim = 100000, 64, 64
    kc, vc, ks, vs, table = make_cache([n], page, 16, 1, dim, seed=11)
    kc.view(torch.uint8).zero_()
    kc[int(table[0, 0]), 0, 0, 0] = 16.0
    ks.fill_(1.0)
    q = torch.zeros(1, 1, dim, device="cuda", dtype=BF)
    q[0, 0, 0] = 1.0
    vc.view(torch.uint8)[int(table[0, 0]), 0] = 0
    vc.copy_(vc.float().abs().to(FP8))
    vs.fill_(2.0 ** -6)
    lens, cu = torch.tensor([n], device="cuda", dtype=torch.int32), torch.tensor([0, 1], device="cuda", dtype=torch.int32)
    want, tol, _ = attention64(q, kc, vc, ks, vs, table, [n], cu, 1.0, 0, False)
    out = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, lens, cu, scale=1.0)
    bounded(out, want, tol, "attention")


def test_attention_strides():
    lens, page, heads, dim = [200, 90], 32, 2, 64
    kc, vc, ks, vs, table = make_cache(lens, page, 8, heads, dim, seed=12)
    cu = torch.tensor([0, 2, 5], device="cuda", dtype=torch.int32)
    kv = torch.tensor(lens, device="cuda", dtype=torch.int32)
    q = rand(5, 4, dim, seed=13)
    want = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu)
    head_major = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc)]
    scales = [s.transpose(1, 2).contiguous().transpose(1, 2) for s in (ks, vs)]
    wide_q = rand(5, 4, dim + 3, seed=14)
    wide_q[..., 1:1 + dim] = q
    wide_out = torch.zeros(5, 4, dim + 5, device="cuda", dtype=BF)
    both = torch.zeros(kc.shape[0], page, 2 * heads, dim, device="cuda", dtype=torch.uint8).view(FP8)
    both[:, :, :heads], both[:, :, heads:] = kc, vc
    wide_table = torch.full((2, table.shape[1] + 3), -5, device="cuda", dtype=torch.int32)
    wide_table[:, :table.shape[1]] = table
    for k, v, a, b in ((*head_major, *scales), (both[:, :, :heads], both[:, :, heads:], ks, vs)):
        got = fp8.paged_attention_fp8(wide_q[..., 1:1 + dim], k, v, a, b, wide_table[:, :table.shape[1]], kv, cu,
                                      out=wide_out[..., 2:2 + dim])
        assert torch.equal(got, want)
    assert bool((wide_out[..., :2] == 0).all()) and bool((wide_out[..., 2 + dim:] == 0).all())


def test_attention_repeats_its_bits():
    for lens, q_lens, width in (([3000, 50, 1200], [1, 1, 1], None), ([500, 300, 400], [200, 100, 90], ROOM // 64)):
        kc, vc, ks, vs, table = make_cache(lens, 64, 16, 4, 128, seed=15, width=width)
        cu = torch.tensor([0, q_lens[0], q_lens[0] + q_lens[1], sum(q_lens)], device="cuda", dtype=torch.int32)
        q, kv = rand(sum(q_lens), 16, 128, seed=16), torch.tensor(lens, device="cuda", dtype=torch.int32)
        first = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu)
        for _ in range(10):
            assert torch.equal(fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu), first)


# ---------------------------------------------------------------------------- streams, graphs, refusals
def test_streams_threads_and_graphs():
    lens = [700, 90, 300]
    kc, vc, ks, vs, table = make_cache(lens, 32, 8, 2, 128, seed=17, width=ROOM // 32)
    kv = torch.tensor(lens, device="cuda", dtype=torch.int32)
    x, (w, sw) = rand(20, 512, seed=18), fp8.quantize_fp8(rand(768, 512, seed=19, std=0.05), 128)

    def both(q, cu, **kw):
        return (fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu, **kw), fp8.gemm_fp8(x, w, sw, **kw))

    one = torch.tensor([0, 1, 2, 3], device="cuda", dtype=torch.int32)
    many = torch.tensor([0, 90, 180, 300], device="cuda", dtype=torch.int32)
    calls = [(rand(3, 8, 128, seed=20), one), (rand(300, 8, 128, seed=21), many)]
    want = [both(*c) for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [both(*c, stream=s) for c, s in zip(calls, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(y, z) for y, z in zip(a, b))
    # two captured graphs, replayed in turn and at once
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(*c)
        graphs.append((g, out))
    for _ in range(3):
        for s, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, a), b in zip(graphs, want):
        assert all(torch.equal(y, z) for y, z in zip(a, b))
    # host threads on one stream
    wrong = []

    def work(c, b):
        for _ in range(30):
            if not all(torch.equal(y, z) for y, z in zip(both(*c), b)):
                wrong.append(c)
    threads = [threading.Thread(target=work, args=(c, b)) for c, b in zip(calls * 2, want * 2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong
    in_order()


def test_python_refusals():
    kc, vc, ks, vs, table = make_cache([40, 30], 16, 8, 2, 64)
    q = rand(2, 4, 64)
    lens, cu = torch.tensor([40, 30], device="cuda", dtype=torch.int32), torch.tensor([0, 1, 2], device="cuda", dtype=torch.int32)
    good = dict(q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, page_table=table, kv_lens=lens, cu_q=cu)
    fp8.paged_attention_fp8(**good)
    for bad in (dict(k_cache=kc.to(BF)), dict(v_cache=vc[:, :8]), dict(k_scale=ks.double()), dict(v_scale=vs[:1]), dict(k_scale=ks.cpu()),
                dict(k_scale=ks[:, :1].expand(-1, 3, -1), v_scale=vs[:, :1].expand(-1, 3, -1)), dict(q=q.float()),
                dict(q=rand(2, 4, 128)), dict(page_table=table.long()), dict(kv_lens=lens[:1]), dict(cu_q=cu[:2]),
                dict(k_cache=kc.transpose(2, 3))):
        with pytest.raises((TypeError, ValueError)):
            fp8.paged_attention_fp8(**{**good, **bad})
    with pytest.raises(layer.LowmError):
        fp8.paged_attention_fp8(**{**good, "q": rand(2, 3, 64)})
    x, w, sw = rand(4, 256), codes(128, 256), torch.ones(1, 2, device="cuda")
    a, sa = fp8.quantize_fp8(x)
    for args in ((x, w.to(BF), sw), (x, w, sw[:, :1]), (x, w[:, :128], sw), (a, w, sw), (x, w, sw, sa), (a, w, sw, sa[:2]),
                 (a.t(), w, sw, sa), (x.float(), w, sw), (x, w.cpu(), sw)):
        with pytest.raises((TypeError, ValueError)):
            fp8.gemm_fp8(*args)
    with pytest.raises(layer.LowmError):
        fp8.gemm_fp8(rand(129, 256), w, sw)
    with pytest.raises(ValueError):
        fp8.quantize_fp8(x, 64)
    with pytest.raises(ValueError):
        fp8.rope_append_fp8(q, q, q, torch.ones(4, 64, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"),
                            torch.zeros(2, dtype=torch.int64, device="cuda"), kc, vc, ks, vs)


def left_in_shared_memory(byte):
    """Leaves `byte` in most of every SM's shared memory: the ring of a product whose weights hold nothing else."""
    w = torch.full((152 * 128, 4096), byte, dtype=torch.uint8, device="cuda").view(FP8)
    a, sa = fp8.quantize_fp8(rand(64, 4096, seed=1))
    fp8.gemm_fp8(a, w, torch.ones(152, 32, device="cuda"), sa)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [1, 4, 16, 64, 128])
@pytest.mark.parametrize("byte", [0x00, 0xbf, 0xff])                # of fp32 words: 0, a negative number, NaN
def test_attention_of_chunks_without_keys(dim, block, byte):
    page = max(block, 16)
    lens, q_lens = [0, -3, 40, 0, 300, 0], [150, 120, 200, 0, 100, 500]
    kc, vc, ks, vs, table = make_cache(lens, page, block, 2, dim, seed=1, width=ROOM // page)
    cu = [sum(q_lens[:i]) for i in range(7)]
    assert widened(6, cu[-1] + 3, 8, 2, dim, page, ROOM // page)
    q = rand(cu[-1] + 3, 8, dim, seed=2)
    kv, cu_q = torch.tensor(lens, device="cuda", dtype=torch.int32), torch.tensor(cu, device="cuda", dtype=torch.int32)
    for window in (0, 50):
        want, tol, lse = attention64(q, kc, vc, ks, vs, table, lens, cu_q, 0.125, window, True)
        for _ in range(3):
            left_in_shared_memory(byte)
            out, got = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu_q, scale=0.125, window=window, return_lse=True)
            bounded(out, want, tol, "attention")
            assert torch.equal(torch.isneginf(got), torch.isneginf(lse)) and not torch.isnan(got).any()
    in_order()


@pytest.mark.parametrize("rows,width", [(3, 4), (700, 4), (700, ROOM // 16)])
def test_attention_of_an_empty_batch_with_many_rows(rows, width):
    kc, vc, ks, vs, table = make_cache([5], 16, 8, 2, 64, width=width)
    none, cu = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = fp8.paged_attention_fp8(rand(rows, 4, 64), kc, vc, ks, vs, table[:0], none, cu, return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("block", [1, 8])
@pytest.mark.parametrize("q_lens,room", [([1, 1], 0), ([400, 300], 0), ([400, 300], ROOM // 8)])
def test_attention_of_lengths_past_the_table(block, q_lens, room):
    # what does not fit the table is not there: the rows stand at the end of what does
    page, wide = 8, bool(room)
    width = room + 3                                                # the last 64 keys' place in the table is not whole
    lens = [width * page + 5, width * page + 60]
    kc, vc, ks, vs, table = make_cache([width * page] * 2, page, block, 2, 64, seed=21)
    cu = [0, q_lens[0], sum(q_lens)]
    assert widened(2, cu[-1], 8, 2, 64, page, width) == wide
    q = rand(cu[-1], 8, 64, seed=22)
    kv, cu_q = torch.tensor(lens, device="cuda", dtype=torch.int32), torch.tensor(cu, device="cuda", dtype=torch.int32)
    layer.release_workspaces()
    junk = torch.full((1 << 28,), 0xff, dtype=torch.uint8, device="cuda")      # memory that a workspace may get
    del junk
    want, tol, lse = attention64(q, kc, vc, ks, vs, table, lens, cu_q, 0.125, 0, wide)
    out, got = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu_q, scale=0.125, return_lse=True)
    bounded(out, want, tol, "attention")
    seen = torch.isfinite(lse)
    assert torch.equal(torch.isneginf(got), ~seen) and float((got[seen] - lse[seen]).abs().max()) <= 1e-3


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [1, 16, 64])
@pytest.mark.parametrize("q_lens,room", [([1, 3], 0), ([40, 30], 0), ([250, 180], 0), ([250, 180], ROOM)])
@pytest.mark.parametrize("window", [0, 60])
def test_attention_value_scales_that_are_none(dim, block, q_lens, room, window):
    # NaN, infinite, negative and too large ones make the rows that see them NaN; those from 0 to 2^-50 count as 2^-50
    lens, page, bad = [400, 260], 64, [math.nan, math.inf, -math.inf, -1.0, 2.0 ** 51, -math.nan]
    kc, vc, ks, vs, table = make_cache(lens, page, block, 2, dim, seed=23, width=room // page if room else None)
    cu = [0, q_lens[0], sum(q_lens)]
    assert widened(2, cu[-1], 8, 2, dim, page, table.shape[1]) == bool(room)
    at = lambda b, key: (int(table[b, key // page]), key % page // block)                  # noqa: E731
    vs[at(0, 130)] = torch.tensor([0.0, 2.0 ** -60], device="cuda")                        # a scale a head
    vs[at(1, 70)] = torch.tensor([2.0 ** -149, 2.0 ** 50], device="cuda")
    for i, key in enumerate((200, 385, 399)):
        vs[at(0, key)] = torch.tensor([bad[2 * i], bad[2 * i + 1]], device="cuda")
    q = rand(cu[-1], 8, dim, seed=24)
    kv, cu_q = torch.tensor(lens, device="cuda", dtype=torch.int32), torch.tensor(cu, device="cuda", dtype=torch.int32)
    taken = (vs >= 0) & (vs <= 2.0 ** 50)
    floor = vs.clamp(min=2.0 ** -50)
    _, tol, _ = attention64(q, kc, vc, ks, torch.where(taken, floor, 1.0), table, lens, cu_q, 0.125, window, bool(room))
    want, _, lse = attention64(q, kc, vc, ks, torch.where(taken, floor, math.nan), table, lens, cu_q, 0.125, window, False)
    out, got = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu_q, scale=0.125, window=window, return_lse=True)
    assert torch.isnan(want).any() and not torch.isnan(want).all()
    bounded(out, want, tol, "attention")
    ok = torch.isfinite(want).all(-1)
    assert float((got[ok] - lse[ok]).abs().max()) <= 1e-3
    in_order()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("batch,kv_heads,room", [(5, 4, 1 << 18), (3, 4, 1 << 20), (2, 2, 1 << 20), (7, 1, 1 << 19)])
@pytest.mark.parametrize("window,block", [(0, 64), (0, 16), (90, 16), (0, 1), (90, 1)])
def test_attention_of_chunks_whose_copies_take_turns(dim, batch, kv_heads, room, window, block):
    # the table has room for far more than the scratch memory: sequences and heads one after the other
    lens = [700, 3, 0, 290, 64, 200, 1000][:batch]
    q_lens = [250, 120, 100, 100, 64, 0, 200][:batch]
    page, heads = 64, 4 * kv_heads
    kc, vc, ks, vs, table = make_cache(lens, page, block, kv_heads, dim, seed=25, width=room // page)
    cu = [3 + sum(q_lens[:i]) for i in range(batch + 1)]
    q = rand(cu[-1] + 5, heads, dim, seed=26)                       # rows of no sequence before and behind
    size = fp8.lowm_paged_attention_fp8_workspace(batch, len(q), heads, kv_heads, dim, page, room // page)
    copies = 4 * batch * kv_heads * room * dim
    assert size > 100 << 20 and size < (1 << 30) + (64 << 20)
    kv, cu_q = torch.tensor(lens, device="cuda", dtype=torch.int32), torch.tensor(cu, device="cuda", dtype=torch.int32)
    want, tol, lse = attention64(q, kc, vc, ks, vs, table[:, :16], lens, cu_q, 0.125, window, True)
    for _ in range(2):
        out, got = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu_q, scale=0.125, window=window, return_lse=True)
        bounded(out, want, tol, "attention of copies of %.1f GiB" % (copies / 2 ** 30))
        seen = torch.isfinite(lse)
        assert torch.equal(torch.isneginf(got), ~seen) and float((got[seen] - lse[seen]).abs().max()) <= 1e-3
    in_order()


@pytest.mark.parametrize("window", [200, 1500])
def test_attention_of_chunks_of_a_long_cache_with_a_window(window):
    # far behind the beginning: the copy holds the window only, in pages that take turns
    check_attention([9000, 20011, 300], [300, 130, 290], 8, 2, 64, 64, 16, window=window, seed=27, width=1 << 14, wide=True)


def test_attention_of_very_many_sequences_in_turns():
    # more of them than a launch has rows of CTAs, and more room in the table than one turn has
    batch, page, room = 1100, 64, 1 << 13
    lens = [(37 * b) % 190 for b in range(batch)]
    q_lens = [0 if b % 9 == 4 else 27 + b % 4 for b in range(batch)]
    kc, vc, ks, vs, table = make_cache(lens, page, 16, 1, 64, seed=30, width=room // page)
    cu = [sum(q_lens[:i]) for i in range(batch + 1)]
    q = rand(cu[-1], 4, 64, seed=31)
    assert widened(batch, cu[-1], 4, 1, 64, page, room // page)
    kv, cu_q = torch.tensor(lens, device="cuda", dtype=torch.int32), torch.tensor(cu, device="cuda", dtype=torch.int32)
    want, tol, lse = attention64(q, kc, vc, ks, vs, table[:, :3], lens, cu, 0.125, 0, True)
    out, got = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu_q, scale=0.125, return_lse=True)
    bounded(out, want, tol, "attention")
    assert torch.equal(torch.isneginf(got), torch.isneginf(lse))
    in_order()


def test_large_workspaces_are_not_kept():
    layer.release_workspaces()
    lens, page = [300], 64
    kc, vc, ks, vs, table = make_cache(lens, page, 16, 8, 128, seed=28, width=1 << 11)
    q = rand(150, 8, 128, seed=29)
    kv, cu = torch.tensor(lens, device="cuda", dtype=torch.int32), torch.tensor([0, 150], device="cuda", dtype=torch.int32)
    assert fp8.lowm_paged_attention_fp8_workspace(1, 150, 8, 8, 128, page, 1 << 11) > 1 << 29
    fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu)
    assert not layer._kept
    fp8.paged_attention_fp8(q[:1], kc, vc, ks, vs, table, kv, torch.tensor([0, 1], device="cuda", dtype=torch.int32))
    assert len(layer._kept) == 1


# The copy has a pair of factors for a tile, for four keys or for a key: each of them at the edges.
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [1, 2, 4, 16, 64])
@pytest.mark.parametrize("window", [0, 30])
def test_attention_of_widened_chunks_with_nan_codes(dim, block, window):
    lens, q_lens, page = [200, 150], [120, 80], 64

    def change(kc, vc, ks, vs, table, q):
        for b, n in enumerate(lens):
            for key, d in ((n - 3, 5), (n - 15, 6), (n - q_lens[b], 7), (n - 40, 8), (2, 9)):
                vc.view(torch.uint8)[int(table[b, key // page]), key % page, 0, d] = 0xff
    out, _ = check_attention(lens, q_lens, 4, 2, dim, page, block, window=window, seed=32, change=change, width=ROOM // page, wide=True)
    assert widened(2, 200, 4, 2, dim, page, ROOM // page) and torch.isnan(out).any() and not torch.isnan(out).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [1, 2, 4, 16, 64])
@pytest.mark.parametrize("window", [0, 30])
def test_attention_of_widened_chunks_where_no_row_sees(dim, block, window):
    lens, q_lens, page = [200, 130, 71, 0], [100, 100, 70, 114], 64
    kc, vc, ks, vs, table = make_cache(lens, page, block, 2, dim, seed=33, width=ROOM // page)
    clean = vs.clone()                                              # the bound multiplies by what is not seen, too
    for b, n in enumerate(lens[:3]):
        last, first_free = int(table[b, (n - 1) // page]), (n - 1) % page + 1
        for c in (kc, vc):
            c.view(torch.uint8)[last, first_free:] = 0x7f
        for s, x in ((ks, math.nan), (vs, -1.0)):
            s[last, -(-first_free // block):] = x
    if window:                                                      # of sequence 0 keys 71 .. are seen
        for c in (kc, vc):
            c.view(torch.uint8)[int(table[0, 0])] = 0xff
        ks[int(table[0, 0])] = math.inf
        vs[int(table[0, 0])] = math.nan
    free = [i for i in range(kc.shape[0]) if i not in [int(p) for b, n in enumerate(lens) for p in table[b, :-(-n // page)]]]
    for c in (kc, vc):
        c.view(torch.uint8)[free] = 0xff
    table[1, 1] = kc.shape[0]                                       # reads as zeros
    cu = [sum(q_lens[:i]) for i in range(5)]
    assert widened(4, cu[-1], 8, 2, dim, page, ROOM // page)
    q = rand(cu[-1], 8, dim, seed=36)
    kv, cu_q = torch.tensor(lens, device="cuda", dtype=torch.int32), torch.tensor(cu, device="cuda", dtype=torch.int32)
    want, tol, lse = attention64(q, kc, vc, ks, clean, table, lens, cu, 0.125, window, True)
    out, got = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu_q, scale=0.125, window=window, return_lse=True)
    bounded(out, want, tol, "attention")
    seen = torch.isfinite(lse)
    assert torch.equal(torch.isneginf(got), ~seen) and float((got[seen] - lse[seen]).abs().max()) <= 1e-3
    in_order()


@pytest.mark.parametrize("block", [1, 16, 64])
@pytest.mark.parametrize("room", [ROOM, 1 << 20])                  # at once, in turns
def test_widened_chunks_repeat_their_bits(block, room):
    lens, q_lens, page = [500, 300, 400], [200, 100, 90], 64
    kc, vc, ks, vs, table = make_cache(lens, page, block, 4, 128, seed=34, width=room // page)
    cu = torch.tensor([0, 200, 300, 390], device="cuda", dtype=torch.int32)
    q, kv = rand(390, 16, 128, seed=35), torch.tensor(lens, device="cuda", dtype=torch.int32)
    assert widened(3, 390, 16, 4, 128, page, room // page)
    first = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu)
    for _ in range(10):
        left_in_shared_memory(0xff)
        assert torch.equal(fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, kv, cu), first)


@pytest.mark.parametrize("window", [0, 100])
def test_a_captured_call_in_turns_follows_the_lengths(window):
    # which sequences share a turn is decided by the device: other lengths, other tables and other rows of q in a replay
    page, room, heads, kv_heads, dim = 64, 1 << 20, 8, 2, 64
    kc, vc, ks, vs, table = make_cache([900, 900, 900, 900], page, 16, kv_heads, dim, seed=37, width=room // page)
    q = rand(400, heads, dim, seed=38)
    kv, cu = (torch.zeros(n, device="cuda", dtype=torch.int32) for n in (4, 5))
    args = (q, kc, vc, ks, vs, table, kv, cu)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fp8.paged_attention_fp8(*args, window=window)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, got = fp8.paged_attention_fp8(*args, window=window, return_lse=True)
    for lens, starts in (([900, 0, 500, 70], [0, 100, 200, 300, 400]), ([0, 0, 0, 900], [0, 0, 0, 1, 390]),
                         ([300, 900, 900, 64], [7, 250, 250, 350, 350]), ([0, 0, 0, 0], [0, 0, 0, 0, 0])):
        kv.copy_(torch.tensor(lens)), cu.copy_(torch.tensor(starts))
        table.copy_(table.roll(1, 0))
        want, tol, lse = attention64(q, kc, vc, ks, vs, table[:, :15], lens, starts, dim ** -0.5, window, True)
        out.fill_(math.nan), got.fill_(math.nan)
        graph.replay()
        bounded(out, want, tol, "attention")
        assert torch.equal(torch.isneginf(got), torch.isneginf(lse)) and not torch.isnan(got).any()
    in_order()


@pytest.mark.parametrize("room", [ROOM, 1 << 20])
def test_chunks_whose_starts_do_not_rise(room):
    # not a call that means anything: sequences whose starts fall have no rows, and the others' are as they would be alone
    page, heads, kv_heads, dim = 64, 8, 2, 64
    kc, vc, ks, vs, table = make_cache([300, 400, 500, 200], page, 16, kv_heads, dim, seed=39, width=room // page)
    q, lens = rand(500, heads, dim, seed=40), torch.tensor([300, 400, 500, 200], device="cuda", dtype=torch.int32)
    cu = torch.tensor([0, 300, 50, 150, 500], device="cuda", dtype=torch.int32)     # sequence 1 falls back; 2 lies in 0's rows
    assert widened(4, 500, heads, kv_heads, dim, page, room // page)
    out = fp8.paged_attention_fp8(q, kc, vc, ks, vs, table, lens, cu)
    alone = torch.tensor([150, 500], device="cuda", dtype=torch.int32)
    want, tol, _ = attention64(q, kc, vc, ks, vs, table[3:, :8], lens[3:], alone, dim ** -0.5, 0, True)
    bounded(out[300:], want[300:], tol[300:], "attention")
    in_order()
