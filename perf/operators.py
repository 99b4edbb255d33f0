"""Measured cases of the decoder-layer operators around the low-M GEMM.

Four operators make up, with the GEMM, one decoder layer for a few tokens:

  norm  residual_norm    r' = scale r + gate * RMS(block; post), n = RMS(r'; pre)
  rope  rope_append      rotary positions (one to three axes) for q and k; k and v go into the paged cache
  attn  paged_attention  a chunk of new tokens (one or many per sequence) against the paged cache
  moe   moe              router, top-k, gated experts and their weighted sum for at most 128 tokens

``run`` computes them in plain torch operations in 32 bits (``own`` false) or
through the package (``own`` true); ``exact`` computes them in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6


# ----------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # The norms around one block while four sequences decode: pure latency.
        {"name": "norm decode", "op": "norm", "tokens": 4, "hidden": 4096, "residual": "bf16", "post": True,
         "gate": "channel", "scale": 1.0},
        # A ragged batch with modulated (per-token) gates, an odd width and a 32-bit residual stream.
        {"name": "norm odd gated", "op": "norm", "tokens": 150, "hidden": 2305, "residual": "f32", "post": True,
         "gate": "token", "scale": 0.5},
        # A long prompt's tokens at once, residual add and next norm only: bandwidth.
        {"name": "norm prompt", "op": "norm", "tokens": 8192, "hidden": 4096, "residual": "bf16", "post": False,
         "gate": "none", "scale": 1.0},
        # Four decoding sequences append one token each.
        {"name": "rope decode", "op": "rope", "tokens": 4, "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "axes": 1, "interleaved": False, "page": 64},
        # A prompt with images (time, height, width positions) enters the cache.
        {"name": "rope prompt 3 axes", "op": "rope", "tokens": 4096, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "axes": 3, "interleaved": False, "page": 16},
        # Four short conversations, one new token each: the latency of a split over few keys.
        {"name": "attn decode short", "op": "attn", "batch": 4, "q_max": 1, "kv_max": 1000, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # A serving batch of very different long contexts, one new token each: bandwidth of the cache.
        {"name": "attn decode long", "op": "attn", "batch": 24, "q_max": 1, "kv_max": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # Verification of drafted tokens (1 to 7 a sequence), small heads and pages, a sliding window.
        {"name": "attn verify window", "op": "attn", "batch": 8, "q_max": 7, "kv_max": 5555, "heads": 64,
         "kv_heads": 8, "dim": 64, "page": 16, "window": 2047},
        # Chunks of two prompts against what their caches already hold: tensor-core bound.
        {"name": "attn chunk", "op": "attn", "batch": 2, "q_max": 1537, "kv_max": 9001, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "window": 0},
        # One token through a layer of many small experts: latency and the bandwidth of 4 experts.
        {"name": "moe single", "op": "moe", "tokens": 1, "hidden": 2048, "inner": 768, "experts": 64, "top_k": 4,
         "scoring": "softmax"},
        # A decode batch that reaches most experts with one or two tokens each.
        {"name": "moe batch", "op": "moe", "tokens": 24, "hidden": 2048, "inner": 768, "experts": 128, "top_k": 8,
         "scoring": "sigmoid"},
        # The largest batch of the low-M regime, wider experts with 16 tokens each on average.
        {"name": "moe 128 tokens", "op": "moe", "tokens": 128, "hidden": 4096, "inner": 1400, "experts": 32,
         "top_k": 4, "scoring": "softmax"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn", "moe", "moe"])
    if op == "norm":
        hidden = rng.choice([_log_int(rng, 257, 4096), 8 * (2 * _log_int(rng, 16, 255) + 1)])
        return {"op": "norm", "tokens": _log_int(rng, 1, 8192), "hidden": hidden,
                "residual": rng.choice(["bf16", "f32"]), "post": rng.random() < 0.6,
                "gate": rng.choice(["none", "channel", "token"]), "scale": rng.choice([1.0, 0.5, 0.7071])}
    if op == "rope":
        dim = rng.choice([64, 128])
        kv = rng.choice([1, 2, 4, 8])
        return {"op": "rope", "tokens": _log_int(rng, 1, 4096), "heads": kv * rng.choice([1, 3, 4]), "kv_heads": kv,
                "dim": dim, "rotary": rng.choice([dim, dim // 2]), "axes": rng.choice([1, 2, 3]),
                "interleaved": rng.random() < 0.5, "page": rng.choice([16, 32, 64])}
    if op == "attn":
        kv = rng.choice([1, 2, 4, 8])
        q_max = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 17, 1200)])
        batch = _log_int(rng, 1, 24 if q_max <= 16 else 3)
        kv_max = _log_int(rng, max(q_max, 17), 16384 if q_max <= 16 else 6000)
        return {"op": "attn", "batch": batch, "q_max": q_max, "kv_max": kv_max,
                "heads": kv * rng.choice([1, 3, 4]), "kv_heads": kv, "dim": rng.choice([64, 128]),
                "page": rng.choice([16, 32, 64, 128]), "window": rng.choice([0, 0, _log_int(rng, 100, 4000)])}
    experts = rng.choice([8, 24, 64, 96])
    return {"op": "moe", "tokens": _log_int(rng, 1, 128), "hidden": 8 * (2 * _log_int(rng, 32, 127) + 1),
            "inner": 8 * (2 * _log_int(rng, 10, 63) + 1), "experts": experts,
            "top_k": rng.choice([1, 2, 5, 8]), "scoring": rng.choice(["softmax", "sigmoid"])}


# ---------------------------------------------------------------------------------------------- inputs
def _lengths(c):
    """Keys (new tokens included) and new tokens of each sequence: part of the case, not of the seed."""
    r = random.Random("%d %d %d" % (c["batch"], c["q_max"], c["kv_max"]))
    q = [c["q_max"]] + [r.randint((c["q_max"] + 1) // 2, c["q_max"]) for _ in range(c["batch"] - 1)]
    kv = [c["kv_max"]] + [max(n, int(c["kv_max"] * r.uniform(0.1, 1.0))) for n in q[1:]]
    return q, kv


def _sections(c):
    half = c["rotary"] // 2
    if c["axes"] == 1:
        return (half,)
    if c["axes"] == 2:
        return (half // 2, half - half // 2)
    a = half // 4
    b = (half - a) // 2
    return (a, b, half - a - b)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return torch.empty(shape, device=dev, dtype=dtype).normal_(mean, std, generator=g)

    s = {"op": c["op"], "case": c}
    if c["op"] == "norm":
        t, h = c["tokens"], c["hidden"]
        rdt = torch.float32 if c["residual"] == "f32" else torch.bfloat16
        s["residual"] = normal(t, h, std=3.0, dtype=rdt)
        s["block"] = normal(t, h, std=0.7)
        s["post"] = normal(h, std=0.1, mean=1.0) if c["post"] else None
        s["gate"] = {"none": None, "channel": (h,), "token": (t, h)}[c["gate"]]
        s["gate"] = normal(*s["gate"], std=0.5) if s["gate"] else None
        s["pre"] = normal(h, std=0.1, mean=1.0)
        s["out_residual"] = torch.empty_like(s["residual"])
        s["out"] = torch.empty_like(s["block"])
    elif c["op"] == "rope":
        t, hq, hk, d = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        s["qkv"] = normal(t, (hq + 2 * hk) * d)          # what the QKV projection wrote
        longest = 32768
        inv = 10000.0 ** (-torch.arange(0, c["rotary"], 2, device=dev, dtype=torch.float64) / c["rotary"])
        ang = torch.arange(longest, device=dev, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        shape = (t,) if c["axes"] == 1 else (c["axes"], t)
        s["positions"] = torch.randint(0, longest, shape, device=dev, generator=g)
        pages = (2 * t + c["page"] - 1) // c["page"] + 1
        s["slots"] = torch.randperm(pages * c["page"], device=dev, generator=g)[:t].contiguous()
        s["k_cache"] = normal(pages, c["page"], hk, d)
        s["v_cache"] = normal(pages, c["page"], hk, d)
        s["sections"] = _sections(c)
        # which axis each rotary pair turns by
        s["axis"] = torch.repeat_interleave(torch.arange(c["axes"], device=dev),
                                            torch.tensor(s["sections"], device=dev))
        s["out"] = torch.empty((t, hq, d), device=dev, dtype=torch.bfloat16)
    elif c["op"] == "attn":
        q_lens, kv_lens = _lengths(c)
        page, b = c["page"], c["batch"]
        per = [(n + page - 1) // page for n in kv_lens]
        pages = sum(per) + 3
        order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
        width = max(per)
        at = torch.tensor([sum(per[:i]) for i in range(b)], device=dev)[:, None] + torch.arange(width, device=dev)
        used = torch.arange(width, device=dev) < torch.tensor(per, device=dev)[:, None]
        s["page_table"] = torch.where(used, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
        s["k_cache"] = normal(pages, page, c["kv_heads"], c["dim"])
        s["v_cache"] = normal(pages, page, c["kv_heads"], c["dim"])
        s["q"] = normal(sum(q_lens), c["heads"], c["dim"], std=1.5)
        s["kv_lens"] = torch.tensor(kv_lens, device=dev, dtype=torch.int32)
        cu = [sum(q_lens[:i]) for i in range(b + 1)]
        s["cu_q"] = torch.tensor(cu, device=dev, dtype=torch.int32)
        s["q_max"] = max(q_lens)
        s["out"] = torch.empty_like(s["q"])
    else:
        t, h, i, e = c["tokens"], c["hidden"], c["inner"], c["experts"]
        s["x"] = normal(t, h)
        s["router"] = normal(e, h, std=1.0 / math.sqrt(h))
        s["bias"] = normal(e, std=0.05, dtype=torch.float32) if c["scoring"] == "sigmoid" else None
        s["gate_up"] = normal(e, 2 * i, h, std=1.0 / math.sqrt(h))
        s["down"] = normal(e, h, i, std=1.0 / math.sqrt(i))
        s["out"] = torch.empty_like(s["x"])
    return s


# --------------------------------------------------------------------------------------------- passes
def run(state):
    return {"norm": _norm, "rope": _rope, "attn": _attn, "moe": _moe}[state["op"]](state)


def _norm(s):
    c = s["case"]
    if own:
        from split_bf16_gemm_swap_gb300 import residual_norm
        return residual_norm(s["residual"], s["block"], post_weight=s["post"], gate=s["gate"], pre_weight=s["pre"],
                             scale=c["scale"], eps=EPS, out_residual=s["out_residual"], out=s["out"])
    y = s["block"].float()
    if s["post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    r = s["residual"].float() * c["scale"] + y
    n = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["pre"].float()
    return r.to(s["residual"].dtype), n.to(torch.bfloat16)


def _split(s):
    c = s["case"]
    t, hq, hk, d = c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    q, k, v = s["qkv"].split([hq * d, hk * d, hk * d], 1)
    return q.view(t, hq, d), k.view(t, hk, d), v.view(t, hk, d)


def _rope(s):
    c = s["case"]
    q, k, v = _split(s)
    if own:
        from split_bf16_gemm_swap_gb300 import rope_append
        rope_append(q, k, v, s["cos_sin"], s["positions"], s["slots"], s["k_cache"], s["v_cache"],
                    sections=s["sections"], interleaved=c["interleaved"], out=s["out"])
        return s["out"], s["k_cache"], s["v_cache"]
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
        return torch.cat([y, x[..., 2 * half:]], -1).to(torch.bfloat16)

    s["k_cache"].view(-1, c["kv_heads"], c["dim"])[s["slots"]] = turned(k)
    s["v_cache"].view(-1, c["kv_heads"], c["dim"])[s["slots"]] = v
    return turned(q), s["k_cache"], s["v_cache"]


def _attn(s):
    c = s["case"]
    if own:
        from split_bf16_gemm_swap_gb300 import paged_attention
        return paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], s["cu_q"],
                               window=c["window"], out=s["out"])
    dev = s["q"].device
    b, hk, d, groups = c["batch"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    table = s["page_table"].long()
    k = s["k_cache"][table].reshape(b, -1, hk, d).float().permute(0, 2, 3, 1)      # [b, hk, d, keys]
    v = s["v_cache"][table].reshape(b, -1, hk, d).float().permute(0, 2, 1, 3)      # [b, hk, keys, d]
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


def _moe(s):
    c = s["case"]
    if own:
        from split_bf16_gemm_swap_gb300 import moe
        return moe(s["x"], s["router"], s["gate_up"], s["down"], c["top_k"], scoring=c["scoring"], bias=s["bias"],
                   out=s["out"])
    x = s["x"].float()
    logits = x @ s["router"].float().t()
    if c["scoring"] == "softmax":
        p = torch.exp(logits - logits.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = torch.sigmoid(logits)
    ids = torch.sort(p if s["bias"] is None else p + s["bias"], dim=-1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = p.gather(1, ids)
    w = w / w.sum(-1, keepdim=True)
    if ids.numel() <= c["experts"]:                        # few choices: their experts' weights, gathered
        gate, up = torch.einsum("tkih,th->tki", s["gate_up"][ids].float(), x).chunk(2, -1)
        y = torch.einsum("tkhi,tki->tkh", s["down"][ids].float(), gate * torch.sigmoid(gate) * up)
        return (y * w[..., None]).sum(1).to(torch.bfloat16)
    share = torch.zeros_like(p).scatter_(1, ids, w)        # many: every expert for every token, and its share
    gate, up = torch.matmul(x, s["gate_up"].float().transpose(1, 2)).chunk(2, -1)
    y = torch.matmul(gate * torch.sigmoid(gate) * up, s["down"].float().transpose(1, 2))
    return torch.einsum("eth,te->th", y, share).to(torch.bfloat16)


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["tokens"] * c["hidden"]
        res = 4 if c["residual"] == "f32" else 2
        size = n * (2 * res + 2 + 2) + 2 * c["hidden"] * (1 + c["post"] + (c["gate"] == "channel"))
        return {"bytes": size + (2 * n if c["gate"] == "token" else 0), "flops": 10 * n}
    if c["op"] == "rope":
        n = c["tokens"] * c["dim"] * (c["heads"] + 2 * c["kv_heads"])
        turned = c["tokens"] * c["rotary"] * (c["heads"] + c["kv_heads"])
        return {"bytes": 4 * n + c["tokens"] * (4 * c["rotary"] + 8 * c["axes"] + 8), "flops": 3 * turned}
    if c["op"] == "attn":
        q_lens, kv_lens = _lengths(c)
        pairs = keys = 0
        for n, kv in zip(q_lens, kv_lens):
            win = c["window"] or kv
            pairs += sum(min(p + 1, win) for p in range(kv - n, kv))
            keys += min(kv, win + n - 1)
        size = 4 * keys * c["kv_heads"] * c["dim"] + 4 * sum(q_lens) * c["heads"] * c["dim"]
        return {"bytes": size, "flops": 4 * c["dim"] * c["heads"] * pairs}
    t, h, i, e, k = c["tokens"], c["hidden"], c["inner"], c["experts"], c["top_k"]
    reached = e * (1 - (1 - k / e) ** t)                   # experts that t tokens reach, on average
    return {"bytes": 6 * reached * h * i + 2 * e * h + 4 * t * h, "flops": 2 * t * e * h + 6 * t * k * h * i}


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """From the definitions, in 64 bits, one row, sequence or expert at a time."""
    c, s = case, prepare(case, seed)
    f = torch.float64
    if c["op"] == "norm":
        r_out, n_out = [], []
        for rows in range(0, c["tokens"], 1024):
            part = slice(rows, rows + 1024)
            y = s["block"][part].to(f)
            if s["post"] is not None:
                y = y / torch.sqrt((y * y).sum(1, keepdim=True) / c["hidden"] + EPS) * s["post"].to(f)
            if s["gate"] is not None:
                y = y * (s["gate"][part] if c["gate"] == "token" else s["gate"]).to(f)
            r = c["scale"] * s["residual"][part].to(f) + y
            r_out.append(r)
            n_out.append(r / torch.sqrt((r * r).sum(1, keepdim=True) / c["hidden"] + EPS) * s["pre"].to(f))
        return torch.cat(r_out), torch.cat(n_out)
    if c["op"] == "rope":
        q, k, v = _split(s)
        half = c["rotary"] // 2
        pos = s["positions"].view(-1, c["tokens"])
        q64, k64 = q.to(f), k.to(f)
        first = 0
        pairs = []
        for axis, n in enumerate(s["sections"]):
            pairs += [(axis, j) for j in range(first, first + n)]
            first += n
        for axis, j in pairs:
            a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
            cos = s["cos_sin"][pos[axis], j].to(f)[:, None]
            sin = s["cos_sin"][pos[axis], half + j].to(f)[:, None]
            for src, dst in ((q, q64), (k, k64)):
                x, y = src[:, :, a].to(f), src[:, :, b].to(f)
                dst[:, :, a] = x * cos - y * sin
                dst[:, :, b] = x * sin + y * cos
        kc, vc = s["k_cache"].to(f), s["v_cache"].to(f)
        kc.view(-1, c["kv_heads"], c["dim"]).index_copy_(0, s["slots"], k64)
        vc.view(-1, c["kv_heads"], c["dim"]).index_copy_(0, s["slots"], v.to(f))
        return q64, kc, vc
    if c["op"] == "attn":
        q_lens, kv_lens = _lengths(c)
        groups = c["heads"] // c["kv_heads"]
        outs, first = [], 0
        for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
            pages = s["page_table"][b, :(kv + c["page"] - 1) // c["page"]].long()
            k = s["k_cache"][pages].flatten(0, 1)[:kv]
            v = s["v_cache"][pages].flatten(0, 1)[:kv]
            at = torch.arange(kv - n, kv, device=k.device)[:, None]
            key = torch.arange(kv, device=k.device)
            hidden = key > at
            if c["window"]:
                hidden = hidden | (key <= at - c["window"])
            heads = []
            for h in range(c["heads"]):
                score = s["q"][first:first + n, h].to(f) @ k[:, h // groups].to(f).t() / math.sqrt(c["dim"])
                heads.append(torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v[:, h // groups].to(f))
            outs.append(torch.stack(heads, 1))
            first += n
        return torch.cat(outs)
    x = s["x"].to(f)
    logits = x @ s["router"].to(f).t()
    p = logits.softmax(-1) if c["scoring"] == "softmax" else 1 / (1 + torch.exp(-logits))
    choice = p if s["bias"] is None else p + s["bias"].to(f)
    ids = torch.sort(choice, dim=-1, descending=True, stable=True)[1][:, :c["top_k"]]
    total = p.gather(1, ids).sum(1)
    out = torch.zeros_like(x)
    for e in range(c["experts"]):
        rows = (ids == e).any(1).nonzero()[:, 0]
        if len(rows):
            hid = x[rows] @ s["gate_up"][e].to(f).t()
            gate, up = hid[:, :c["inner"]], hid[:, c["inner"]:]
            hid = gate / (1 + torch.exp(-gate)) * up
            out[rows] += (hid @ s["down"][e].to(f).t()) * (p[rows, e] / total[rows])[:, None]
    return out
