"""Measured cases of decoding in 8 bits: weights, key/value cache and its pages.

Next to the bf16 GEMM and the decoder-layer operators stand their 8-bit forms
(e4m3 codes with fp32 scales) and the operators that share the pages of a cache:

  gemm     gemm_fp8             C = A W^T; A bf16, quantised by token and 128 columns, W in blocks of 128 x 128
  append   rope_append_fp8      rotary positions; k and v into a cache of codes with a scale by block of tokens and head
  attn     paged_attention_fp8  a chunk of new tokens (one or many per sequence) against that cache
  fork     fork_pages, copy_pages, extend_pages   one step of a beam search: rows follow their parents
  compact  compact_pages, copy_pages              the used pages move to the front of the pool

``run`` computes them in plain torch operations in 32 bits (``own`` false) or
through the package (``own`` true); ``exact`` computes them in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
LARGEST = 448.0                    # of e4m3


# ----------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # A projection while four sequences decode: the smallest batch, the bandwidth of the weights.
        {"name": "gemm decode", "op": "gemm", "m": 4, "n": 6144, "k": 4096},
        # A ragged batch through a small layer: no size a multiple of its block.
        {"name": "gemm ragged", "op": "gemm", "m": 37, "n": 2311, "k": 1360},
        # The vocabulary's projection of the largest batch: as many activation bytes a tile as weights.
        {"name": "gemm 128 tokens wide", "op": "gemm", "m": 128, "n": 49152, "k": 4096},
        # Four decoding sequences append one token each, in the middle of a block of scales.
        {"name": "append decode", "op": "append", "batch": 4, "new_max": 1, "start_max": 3000, "heads": 32, "kv_heads": 8,
         "dim": 128, "rotary": 128, "axes": 1, "interleaved": False, "page": 64, "block": 16},
        # Chunks of three prompts with images (time, height, width positions) enter the cache.
        {"name": "append prompt 3 axes", "op": "append", "batch": 3, "new_max": 1501, "start_max": 2000, "heads": 32,
         "kv_heads": 8, "dim": 128, "rotary": 128, "axes": 3, "interleaved": False, "page": 16, "block": 16},
        # Four short conversations, one new token each: the latency of a split over few keys.
        {"name": "attn decode short", "op": "attn", "batch": 4, "q_max": 1, "kv_max": 1000, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "block": 16, "window": 0},
        # A serving batch of very different long contexts, one new token each: bandwidth of the cache.
        {"name": "attn decode long", "op": "attn", "batch": 24, "q_max": 1, "kv_max": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "block": 16, "window": 0},
        # Verification of drafted tokens (1 to 7 a sequence), small heads and pages, a sliding window.
        {"name": "attn verify window", "op": "attn", "batch": 8, "q_max": 7, "kv_max": 5555, "heads": 64,
         "kv_heads": 8, "dim": 64, "page": 16, "block": 8, "window": 2047},
        # Chunks of two prompts against what their caches already hold: tensor-core bound.
        {"name": "attn chunk", "op": "attn", "batch": 2, "q_max": 1537, "kv_max": 9001, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "block": 64, "window": 0},
        # Two requests of four beams each after a step: tables, a handful of pages to copy, the next token's place.
        {"name": "fork few beams", "op": "fork", "groups": 2, "beams": 4, "len_max": 1500, "page": 64, "block": 16,
         "layers": 4, "kv_heads": 8, "dim": 128, "spare": 40},
        # A batch of sixteen requests of eight beams: page copies of all layers.
        {"name": "fork many beams", "op": "fork", "groups": 16, "beams": 8, "len_max": 2000, "page": 32, "block": 32,
         "layers": 8, "kv_heads": 4, "dim": 128, "spare": 300},
        # Half of the requests of a pool have ended; the pages of the others are brought together.
        {"name": "compact pool", "op": "compact", "pages": 4096, "rows": 41, "page": 16, "block": 16, "layers": 4,
         "kv_heads": 8, "dim": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "append", "attn", "attn", "fork", "compact"])
    if op == "gemm":
        return {"op": "gemm", "m": _log_int(rng, 1, 128), "n": _log_int(rng, 65, 20001), "k": 16 * _log_int(rng, 5, 700)}
    kv = rng.choice([1, 2, 4, 8])
    if op in ("append", "attn"):
        page = rng.choice([16, 32, 64, 128])
        c = {"op": op, "heads": kv * rng.choice([1, 3, 4]), "kv_heads": kv, "dim": rng.choice([64, 128]), "page": page,
             "block": rng.choice([b for b in (1, 8, 16, 32, 64) if b <= page])}
        if op == "append":
            new = rng.choice([1, _log_int(rng, 2, 16), _log_int(rng, 17, 1400)])
            c.update(batch=_log_int(rng, 1, 64 if new <= 16 else 3), new_max=new, start_max=_log_int(rng, 1, 4000),
                     rotary=rng.choice([c["dim"], c["dim"] // 2]), axes=rng.choice([1, 2, 3]),
                     interleaved=rng.random() < 0.5)
        else:
            q_max = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 1200)])
            c.update(q_max=q_max, batch=_log_int(rng, 1, 24 if q_max <= 16 else 3),
                     kv_max=_log_int(rng, max(q_max, 17), 16384 if q_max <= 16 else 6000),
                     window=rng.choice([0, 0, _log_int(rng, 100, 4000)]))
        return c
    page = rng.choice([16, 32, 64])
    c = {"op": op, "page": page, "block": rng.choice([8, 16]), "layers": rng.randint(1, 6), "kv_heads": kv,
         "dim": rng.choice([64, 128])}
    if op == "fork":
        c.update(groups=_log_int(rng, 1, 16), beams=rng.randint(1, 8), len_max=_log_int(rng, 20, 2000),
                 spare=rng.choice([0, 5, 150]))
    else:
        c.update(pages=_log_int(rng, 60, 4000), rows=_log_int(rng, 1, 50))
    return c


# ---------------------------------------------------------------------------------------------- inputs
def _lengths(c):
    """Keys (new tokens included) and new tokens of each sequence: part of the case, not of the seed."""
    r = random.Random("%d %d %d" % (c["batch"], c["q_max"], c["kv_max"]))
    q = [c["q_max"]] + [r.randint((c["q_max"] + 1) // 2, c["q_max"]) for _ in range(c["batch"] - 1)]
    kv = [c["kv_max"]] + [max(n, int(c["kv_max"] * r.uniform(0.1, 1.0))) for n in q[1:]]
    return q, kv


def _starts(c):
    """Tokens that each sequence has and those that it appends."""
    r = random.Random("%d %d %d" % (c["batch"], c["new_max"], c["start_max"]))
    new = [c["new_max"]] + [r.randint((c["new_max"] + 1) // 2, c["new_max"]) for _ in range(c["batch"] - 1)]
    return [r.randint(0, c["start_max"]) for _ in new], new


def _sections(c):
    half = c["rotary"] // 2
    if c["axes"] == 1:
        return (half,)
    if c["axes"] == 2:
        return (half // 2, half - half // 2)
    a = half // 4
    b = (half - a) // 2
    return (a, b, half - a - b)


def _beam_rows(c):
    """Tokens of each row before the step and its parent; the rows of a request share their prompt."""
    r = random.Random("%d %d %d" % (c["groups"], c["beams"], c["len_max"]))
    prompts = [c["len_max"] // 2 if g == 0 else r.randint(1, max(1, c["len_max"] // 2)) for g in range(c["groups"])]
    lens, parents = [], []
    for g, prompt in enumerate(prompts):
        n = min(c["len_max"], prompt + r.randint(1, max(1, c["len_max"] // 2)))
        lens += [n] * c["beams"]
        parents += [g * c["beams"] + r.randrange(c["beams"]) for _ in range(c["beams"])]
    if c["groups"] > 2:                                   # one request has ended
        parents[-c["beams"]:] = [-1] * c["beams"]
    return prompts, lens, parents


def _pool_rows(c):
    """Tokens of the rows that are left in a pool: about half of its pages."""
    r = random.Random("%d %d %d" % (c["pages"], c["rows"], c["page"]))
    each = max(1, c["pages"] * c["page"] // (2 * c["rows"]))
    return [r.randint((each + 1) // 2, each) for _ in range(min(c["rows"], c["pages"] // 2))]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.empty(shape, device=dev, dtype=dtype).normal_(mean, std, generator=g)

    def codes(*shape):
        return normal(*shape, std=100.0).clamp_(-LARGEST, LARGEST).to(FP8)

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, device=dev, dtype=dtype)

    s = {"op": c["op"], "case": c}
    if c["op"] == "gemm":
        s["a"] = normal(c["m"], c["k"])
        blocks = ((c["n"] + 127) // 128, (c["k"] + 127) // 128)
        s["w"] = codes(c["n"], c["k"])
        s["w_scale"] = torch.empty(blocks, device=dev).uniform_(0.5, 1.5, generator=g) * (0.01 / math.sqrt(c["k"]))
        s["out"] = torch.empty((c["m"], c["n"]), device=dev, dtype=torch.bfloat16)
        return s

    hk, d, page, block = c["kv_heads"], c["dim"], c["page"], c["block"]

    def cache(*pages):
        """Codes and scales; powers of two, as the append leaves them."""
        scale = torch.exp2(torch.randint(-8, -5, (*pages, page // block, hk), device=dev, generator=g).float())
        return codes(*pages, page, hk, d), scale

    if c["op"] in ("append", "attn"):
        if c["op"] == "append":
            start, new = _starts(c)
            total = [a + n for a, n in zip(start, new)]
        else:
            new, total = _lengths(c)
        batch = len(new)
        per = [(n + page - 1) // page for n in total]
        pages = sum(per) + 3
        order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
        width = max(per)
        at = ints([sum(per[:i]) for i in range(batch)], torch.int64)[:, None] + torch.arange(width, device=dev)
        used = torch.arange(width, device=dev) < ints(per, torch.int64)[:, None]
        table = torch.where(used, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
        cu = [sum(new[:i]) for i in range(batch + 1)]
        s["cu_q"] = ints(cu)
        s["k_cache"], s["k_scale"] = cache(pages)
        s["v_cache"], s["v_scale"] = cache(pages)
    if c["op"] == "append":
        t, hq = cu[-1], c["heads"]
        s["qkv"] = normal(t, (hq + 2 * hk) * d)            # what the QKV projection wrote
        longest = 32768
        inv = 10000.0 ** (-torch.arange(0, c["rotary"], 2, device=dev, dtype=torch.float64) / c["rotary"])
        ang = torch.arange(longest, device=dev, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        row = torch.arange(t, device=dev)
        seq = torch.searchsorted(s["cu_q"][1:].long(), row, right=True)
        pos = ints(start, torch.int64)[seq] + row - s["cu_q"].long()[seq]
        s["slots"] = table[seq, pos // page].long() * page + pos % page
        s["positions"] = pos if c["axes"] == 1 else torch.cat(
            [pos[None], torch.randint(0, longest, (c["axes"] - 1, t), device=dev, generator=g)])
        s["sections"] = _sections(c)
        s["axis"] = torch.repeat_interleave(torch.arange(c["axes"], device=dev), ints(s["sections"], torch.int64))
        s["out"] = torch.empty((t, hq, d), device=dev, dtype=torch.bfloat16)
    elif c["op"] == "attn":
        s["page_table"] = table
        for name in ("k_scale", "v_scale"):                # a scale need not be a power of two
            s[name] *= torch.empty_like(s[name]).uniform_(0.6, 1.2, generator=g)
        s["q"] = normal(cu[-1], c["heads"], d, std=1.5)
        s["kv_lens"] = ints(total)
        s["q_max"] = max(new)
        s["out"] = torch.empty_like(s["q"])
    elif c["op"] == "fork":
        prompts, lens, parents = _beam_rows(c)
        rows, beams = len(lens), c["beams"]
        width = (c["len_max"] + page - 1) // page + 1
        ids, entries = [], 0                               # a row's pages, numbered before the shuffle
        for i, n in enumerate(lens):
            shared = prompts[i // beams] // page           # whole pages of the prompt
            first = entries if i % beams == 0 else ids[i - i % beams][0] if shared else entries
            own_from = entries + shared if i % beams == 0 else entries
            need = (n + page - 1) // page
            line = [first + j for j in range(shared)] + [own_from + j for j in range(need - shared)]
            entries = max(entries, own_from + need - shared)
            ids.append(line)
        pages = entries + c["spare"]
        order = torch.randperm(pages, device=dev, generator=g)
        flat = ints([line + [-1] * (width - len(line)) for line in ids], torch.int64)
        s["page_table"] = torch.where(flat >= 0, order[flat.clamp(min=0)], -1).to(torch.int32)
        s["lens"], s["parents"], s["cu_new"] = ints(lens), ints(parents), ints([0] * (rows + 1))
        live = [p >= 0 for p in parents]
        s["cu_new"] = ints([sum(live[:i]) for i in range(rows + 1)])     # one new token for each row that goes on
        s["tokens"] = sum(live)
        s["refs"] = torch.zeros(pages, device=dev, dtype=torch.int32).index_add_(
            0, s["page_table"].flatten().clamp(min=0), (flat >= 0).int().flatten())
        s["caches"] = [*cache(c["layers"], pages), *cache(c["layers"], pages)]
    else:
        lens = _pool_rows(c)
        need = [(n + page - 1) // page for n in lens]
        width = max(need) + 1
        order = torch.randperm(c["pages"], device=dev, generator=g)
        flat = ints([[sum(need[:i]) + j if j < n else -1 for j in range(width)] for i, n in enumerate(need)], torch.int64)
        s["page_table"] = torch.where(flat >= 0, order[flat.clamp(min=0)], -1).to(torch.int32)
        s["lens"] = ints(lens)
        s["refs"] = torch.zeros(c["pages"], device=dev, dtype=torch.int32).index_add_(
            0, s["page_table"].flatten().clamp(min=0), (flat >= 0).int().flatten())
        s["caches"] = [*cache(c["layers"], c["pages"]), *cache(c["layers"], c["pages"])]
    if "caches" in s:
        s["views"] = [x for stacked in s["caches"] for x in stacked.unbind(0)]           # one tensor of a layer each
    return s


# --------------------------------------------------------------------------------------------- passes
def run(state):
    return {"gemm": _gemm, "append": _append, "attn": _attn, "fork": _fork, "compact": _compact}[state["op"]](state)


def _power_of_two(amax):
    """The smallest power of two that brings amax (at least 2^-91) to 448 or less, and its inverse."""
    mantissa, exponent = torch.frexp(amax)
    e = (exponent - 9 + (mantissa > 0.875)).clamp(min=-100)
    e = torch.where(amax > 0, e, -100).to(torch.int32)
    return ((e + 127) << 23).view(torch.float32), ((127 - e) << 23).view(torch.float32)


def _gemm(s):
    c = s["case"]
    if own:
        from split_bf16_gemm_swap_gb300 import gemm_fp8
        return gemm_fp8(s["a"], s["w"], s["w_scale"], out=s["out"])
    n, k = c["n"], c["k"]
    kb = (k + 127) // 128
    a = torch.nn.functional.pad(s["a"].float(), (0, kb * 128 - k)).view(-1, kb, 128)
    scale, inverse = _power_of_two(a.abs().amax(-1, keepdim=True))
    a = ((a * inverse).to(FP8).float() * scale).view(-1, kb * 128)[:, :k]
    w_scale = s["w_scale"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return (a @ (s["w"].float() * w_scale).t()).to(torch.bfloat16)


def _split(s):
    c = s["case"]
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    q, k, v = s["qkv"].split([hq * d, hk * d, hk * d], 1)
    return q.view(-1, hq, d), k.view(-1, hk, d), v.view(-1, hk, d)


def _append(s):
    c = s["case"]
    q, k, v = _split(s)
    if own:
        from split_bf16_gemm_swap_gb300 import rope_append_fp8
        rope_append_fp8(q, k, v, s["cos_sin"], s["positions"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"],
                        s["v_scale"], sections=s["sections"], interleaved=c["interleaved"], out=s["out"])
        return s["out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    half = c["rotary"] // 2
    if c["axes"] == 1:
        rows = s["cos_sin"][s["positions"]]
        cos, sin = rows[:, None, :half], rows[:, None, half:]
    else:
        pos = s["positions"].t()[:, s["axis"]]
        pair = torch.arange(half, device=pos.device)
        cos, sin = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, pair + half][:, None]

    def turned(x):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([y, x[..., 2 * half:]], -1)

    block, hk, d = c["block"], c["kv_heads"], c["dim"]
    at = s["slots"] // block                               # a token's block of scales
    first = s["slots"][s["cu_q"][:-1].long()]              # where each sequence goes on
    first_at, older = first // block, (first % block)[:, None]

    def put(x, cache, scales):
        scales, cells = scales.view(-1, hk), cache.view(torch.uint8).view(-1, block, hk, d)
        amax = x.abs().amax(-1)
        top = torch.zeros_like(scales).scatter_reduce_(0, at[:, None].expand_as(amax), amax, "amax")
        now = _power_of_two(top)[0]
        before = scales[first_at]                          # older tokens of a block that goes on keep their share
        now[first_at] = torch.maximum(now[first_at], torch.where(older > 0, before, 0.0))
        kept = cells[first_at]
        again = (kept.view(FP8).float() * (before / now[first_at])[:, None, :, None]).to(FP8).view(torch.uint8)
        old = torch.arange(block, device=x.device) < older
        cells[first_at] = torch.where(old[:, :, None, None], again, kept)
        scales[at] = now[at]
        cells.view(-1, hk, d)[s["slots"]] = (x / now[at][..., None]).to(FP8).view(torch.uint8)

    put(turned(k), s["k_cache"], s["k_scale"])
    put(v.float(), s["v_cache"], s["v_scale"])
    return turned(q).to(torch.bfloat16), s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _attn(s):
    c = s["case"]
    if own:
        from split_bf16_gemm_swap_gb300 import paged_attention_fp8
        return paged_attention_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["page_table"],
                                   s["kv_lens"], s["cu_q"], window=c["window"], out=s["out"])
    dev = s["q"].device
    b, hk, d, groups = c["batch"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    table = s["page_table"].long()

    def values(cache, scale):                              # [b, keys, hk, d]
        x = cache.view(torch.uint8)[table].view(FP8).float()
        return (x * scale[table].repeat_interleave(c["block"], 2)[..., None]).reshape(b, -1, hk, d)

    k = values(s["k_cache"], s["k_scale"]).permute(0, 2, 3, 1)                      # [b, hk, d, keys]
    v = values(s["v_cache"], s["v_scale"]).permute(0, 2, 1, 3)                      # [b, hk, keys, d]
    q_len, kv_len = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), s["kv_lens"].long()
    step = torch.arange(s["q_max"], device=dev)
    token = (s["cu_q"][:-1].long()[:, None] + step).clamp(max=s["q"].shape[0] - 1)  # padded to the longest chunk
    q = s["q"][token].float().view(b, -1, hk, groups, d).permute(0, 2, 1, 3, 4).reshape(b, hk, -1, d)
    p = torch.matmul(q * (1.0 / math.sqrt(d)), k).view(b, hk, -1, groups, k.shape[-1])
    pos = (kv_len - q_len)[:, None] + step                                          # [b, q_max]
    key = torch.arange(k.shape[-1], device=dev)
    seen = (key <= pos[..., None]) & (pos[..., None] < kv_len[:, None, None])
    if c["window"]:
        seen &= key > pos[..., None] - c["window"]
    p.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    p -= p.amax(-1, keepdim=True).clamp(min=-1e30)
    p.exp_()
    p /= p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.flatten(2, 3), v).view(b, hk, -1, groups, d).permute(0, 2, 1, 3, 4).reshape(b, -1, hk * groups, d)
    row = torch.arange(s["q"].shape[0], device=dev)
    seq = torch.searchsorted(s["cu_q"][1:], row.to(torch.int32), right=True)
    return o[seq, row - s["cu_q"][seq]].to(torch.bfloat16)


def _copied(caches, src, dst):
    chosen = dst >= 0
    src, dst = src[chosen].long(), dst[chosen].long()
    for stacked in caches:
        cells = stacked.view(torch.uint8)
        cells[:, dst] = cells[:, src]


def _fork(s):
    c = s["case"]
    page = c["page"]
    refs = s["refs"].clone()                               # a pass changes them
    if own:
        from split_bf16_gemm_swap_gb300 import copy_pages, extend_pages, fork_pages
        table, lens, src, dst, missing = fork_pages(s["page_table"], s["lens"], s["parents"], refs, page)
        copy_pages(s["views"], src, dst)
        positions, slots, short = extend_pages(table, lens, s["cu_new"], refs, page, s["tokens"])
        return table, lens, refs, src, dst, missing, positions, slots, short, s["caches"]
    dev, old = refs.device, s["page_table"]
    rows, width = s["parents"].shape[0], old.shape[1]
    column, line = torch.arange(width, device=dev), torch.arange(rows, device=dev)

    def taken(ranked, refs):
        """The ranked-th free page, or -1 when there are fewer; and how many there are."""
        full = (refs != 0).int()
        free = torch.sort(full, stable=True)[1].int()
        count = refs.shape[0] - full.sum()
        return torch.where(ranked < count, free[ranked.clamp(0, refs.shape[0] - 1)], -1), count

    parent, goes_on = s["parents"].long().clamp(min=0), s["parents"] >= 0
    lens = torch.where(goes_on, s["lens"][parent], 0)
    count_of = lambda n: (n + page - 1) // page            # noqa: E731
    table = torch.where(column < count_of(lens)[:, None], old[parent], -1)
    for entries, sign, n in ((old, -1, s["lens"]), (table, 1, lens)):
        counted = ((column < count_of(n)[:, None]) & (entries >= 0)).int()
        refs.index_add_(0, entries.clamp(min=0).flatten(), sign * counted.flatten())
    # Rows that share an unfinished last page: the first keeps it.
    last = (count_of(lens) - 1).clamp(min=0)
    tail = torch.where(lens % page != 0, table[line, last], -1)
    again = ((tail[:, None] == tail) & (line < line[:, None])).any(1) & (tail >= 0)
    page_of, free = taken(again.cumsum(0) - again.long(), refs)
    missing = (again.sum() - free).clamp(min=0).int().view(1)
    again = again & (page_of >= 0)
    src, dst = torch.where(again, tail, -1), torch.where(again, page_of, -1)
    table[line, last] = torch.where(again, dst, table[line, last])
    refs.index_add_(0, dst.clamp(min=0), again.int())
    refs.index_add_(0, src.clamp(min=0), -again.int())
    _copied(s["caches"], src, dst)
    # New tokens: pages for those that begin one.
    new = s["cu_new"][1:] - s["cu_new"][:-1]
    before, after = count_of(lens), count_of(lens + new)
    begins = (column >= before[:, None]) & (column < after[:, None])
    ranked = (begins.flatten().cumsum(0) - begins.flatten().long()).view_as(begins)
    page_of, free = taken(ranked, refs)
    short = (begins.sum() - free).clamp(min=0).int().view(1)
    table = torch.where(begins, page_of, table)
    refs.index_add_(0, table.clamp(min=0).flatten(), (begins & (table >= 0)).int().flatten())
    token = torch.arange(s["tokens"], device=dev)
    seq = torch.searchsorted(s["cu_new"][1:], token.to(torch.int32), right=True)
    positions = lens[seq].long() + token - s["cu_new"][seq].long()
    on = table[seq, positions // page].long()
    slots = torch.where(on >= 0, on * page + positions % page, -1)
    return table, lens + new, refs, src, dst, missing, positions, slots, short, s["caches"]


def _compact(s):
    refs, table = s["refs"].clone(), s["page_table"].clone()
    if own:
        from split_bf16_gemm_swap_gb300 import compact_pages, copy_pages
        src, dst, used = compact_pages(table, s["lens"], refs, s["case"]["page"])
        copy_pages(s["views"], src, dst)
        return table, refs, src, dst, used, s["caches"]
    n = refs.shape[0]
    place = torch.arange(n, device=refs.device)
    full = refs != 0
    used = full.sum()
    moves, holes = full & (place >= used), ~full & (place < used)

    def packed(chosen):                                    # the chosen places in order, then -1
        to = torch.where(chosen, chosen.cumsum(0) - 1, n // 2)
        return torch.full((n // 2 + 1,), -1, device=refs.device).scatter_(0, to, torch.where(chosen, place, -1))[:n // 2]

    src, dst = packed(moves), packed(holes)
    rank = (moves.cumsum(0) - 1).clamp(min=0)
    goes = torch.where(moves, dst[rank.clamp(max=n // 2 - 1)], place)
    counted = torch.arange(table.shape[1], device=refs.device) < ((s["lens"] + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    counted &= table >= 0
    table = torch.where(counted, goes[table.clamp(min=0).long()], table).int()
    left = torch.where(moves, 0, refs)
    refs = left.index_add_(0, goes, torch.where(moves, refs, 0))
    _copied(s["caches"], src, dst)
    return table, refs, src.int(), dst.int(), used.int().view(1), s["caches"]


def work(case):
    c = case
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": n * k + 2 * m * k + 2 * m * n + 4 * ((n + 127) // 128) * ((k + 127) // 128), "flops": 2 * m * n * k}
    if c["op"] == "append":
        start, new = _starts(c)
        t = sum(new)
        scales = 8 * c["kv_heads"] * sum((a + n - 1) // c["block"] - a // c["block"] + 1 for a, n in zip(start, new))
        kept = 4 * c["kv_heads"] * c["dim"] * sum(a % c["block"] for a in start)
        size = t * c["dim"] * (4 * c["heads"] + 6 * c["kv_heads"]) + t * (4 * c["rotary"] + 8 * c["axes"] + 8)
        return {"bytes": size + scales + kept, "flops": 3 * t * c["rotary"] * (c["heads"] + c["kv_heads"])}
    if c["op"] == "attn":
        q_lens, kv_lens = _lengths(c)
        pairs = keys = 0
        for n, kv in zip(q_lens, kv_lens):
            win = c["window"] or kv
            pairs += sum(min(p + 1, win) for p in range(kv - n, kv))
            keys += min(kv, win + n - 1)
        size = 2 * keys * c["kv_heads"] * (c["dim"] + 4 / c["block"]) + 4 * sum(q_lens) * c["heads"] * c["dim"]
        return {"bytes": size, "flops": 4 * c["dim"] * c["heads"] * pairs}
    one = 2 * c["layers"] * c["kv_heads"] * (c["page"] * c["dim"] + 4 * c["page"] // c["block"])   # a page's bytes
    if c["op"] == "fork":
        _, lens, parents = _beam_rows(c)
        need = lambda n: (n + c["page"] - 1) // c["page"]  # noqa: E731
        rows = [lens[p] for p in parents if p >= 0]
        copies = sum(1 for i, p in enumerate(parents) if p >= 0 and lens[p] % c["page"] and p in parents[:i])
        entries = sum(map(need, lens)) + sum(map(need, rows))
        return {"bytes": 2 * copies * one + 12 * entries + 24 * len(rows), "flops": 0}
    need = [(n + c["page"] - 1) // c["page"] for n in _pool_rows(c)]
    moves = sum(need) * (c["pages"] - sum(need)) / c["pages"]          # on average
    return {"bytes": 2 * moves * one + 12 * c["pages"] + 8 * sum(need), "flops": 0}


# ------------------------------------------------------------------------------------------ in 64 bits
def _rounded(x):
    """The nearest values of 4 significant bits, at least 2^-9 apart (e4m3), ties to the even one; |x| <= 448."""
    f = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    step = torch.pow(2.0, f - 3)
    return torch.round(x / step) * step


def _scale64(amax):
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / LARGEST)).clamp(min=-100)
    e = torch.where(LARGEST * torch.pow(2.0, e - 1) >= amax, e - 1, e)
    e = torch.where(LARGEST * torch.pow(2.0, e) < amax, e + 1, e).clamp(min=-100)
    return torch.pow(2.0, e)


def exact(case, seed):
    """From the definitions, in 64 bits, one row, sequence or head at a time.  Pages and their tables are whole numbers."""
    c = case
    if c["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    f = torch.float64
    if c["op"] == "gemm":
        a, out = s["a"].to(f), torch.zeros((c["m"], c["n"]), device=s["a"].device, dtype=f)
        for j, k0 in enumerate(range(0, c["k"], 128)):
            part = a[:, k0:k0 + 128]
            scale = _scale64(part.abs().amax(1, keepdim=True))
            part = _rounded(part / scale) * scale
            row = s["w_scale"][:, j].to(f)
            product = part @ s["w"][:, k0:k0 + 128].to(f).t()
            for i in range(row.shape[0]):
                out[:, 128 * i:128 * i + 128] += product[:, 128 * i:128 * i + 128] * row[i]
        return out
    hk, d, block = c["kv_heads"], c["dim"], c["block"]
    if c["op"] == "append":
        q, k, v = _split(s)
        half, t = c["rotary"] // 2, s["slots"].shape[0]
        pos = s["positions"].view(-1, t)
        q64, k64 = q.to(f), k.to(f)
        first, pairs = 0, []
        for axis, n in enumerate(s["sections"]):
            pairs += [(axis, j) for j in range(first, first + n)]
            first += n
        for axis, j in pairs:
            a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
            cos = s["cos_sin"][pos[axis], j].to(f)[:, None]
            sin = s["cos_sin"][pos[axis], half + j].to(f)[:, None]
            for src, to in ((q, q64), (k, k64)):
                x, y = src[:, :, a].to(f), src[:, :, b].to(f)
                to[:, :, a] = x * cos - y * sin
                to[:, :, b] = x * sin + y * cos
        out = []
        cu, slots = s["cu_q"].tolist(), s["slots"].tolist()
        for x, cache, scale in ((k64, s["k_cache"], s["k_scale"]), (v.to(f), s["v_cache"], s["v_scale"])):
            cells, scale = cache.to(f).view(-1, hk, d), scale.to(f).view(-1, hk)
            for b in range(c["batch"]):
                t0 = cu[b]
                while t0 < cu[b + 1]:                      # the tokens of one block of scales
                    place = slots[t0] % block
                    n = min(block - place, cu[b + 1] - t0)
                    at, line = slots[t0] // block, slots[t0] - place
                    now = _scale64(x[t0:t0 + n].abs().amax((0, 2)))
                    if place:
                        now = torch.maximum(now, scale[at])
                        older = cells[line:line + place] * (scale[at] / now)[:, None]
                        cells[line:line + place] = _rounded(older)
                    cells[line + place:line + place + n] = _rounded(x[t0:t0 + n] / now[:, None])
                    scale[at] = now
                    t0 += n
            out += [cells.view(cache.shape), scale.view(s["k_scale"].shape)]
        return q64, out[0], out[2], out[1], out[3]
    q_lens, kv_lens = _lengths(c)
    groups, page = c["heads"] // hk, c["page"]
    outs, first = [], 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        pages = s["page_table"][b, :(kv + page - 1) // page].tolist()
        gathered = []
        for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
            x = torch.cat([cache[i:i + 1] for i in pages]).to(f).view(-1, block, hk, d)
            by = torch.cat([scale[i:i + 1] for i in pages]).to(f).view(-1, 1, hk, 1)
            gathered.append((x * by).view(-1, hk, d)[:kv])
        k, v = gathered
        at = torch.arange(kv - n, kv, device=k.device)[:, None]
        key = torch.arange(kv, device=k.device)
        hidden = key > at
        if c["window"]:
            hidden = hidden | (key <= at - c["window"])
        heads = []
        for h in range(c["heads"]):
            score = s["q"][first:first + n, h].to(f) @ k[:, h // groups].t() / math.sqrt(d)
            heads.append(torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v[:, h // groups])
        outs.append(torch.stack(heads, 1))
        first += n
    return torch.cat(outs)
