"""A small mixture-of-experts decoder run from end to end on the library's operators.

Four prompts of different lengths go through the layers as one ragged chunk,
then every sequence decodes greedily, one token a step: the projections on the
low-M GEMM, everything between them on the decoder-layer operators.  Weights
are random; there is no tokenizer.

    python examples/decoder_layer.py            # prints the tokens and the time of a step
    python examples/decoder_layer.py --check    # also compares every step with plain torch
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from split_bf16_gemm_swap_gb300 import gemm, moe, paged_attention, residual_norm, rope_append  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, ROTARY = 1024, 16, 4, 64, 64
EXPERTS, TOP_K, INNER, LAYERS, VOCAB = 16, 2, 512, 3, 2048
PAGE, MAX_POSITION, EPS, BRANCH = 16, 1024, 1e-6, 0.5
BF = torch.bfloat16


def make_weights(seed: int = 0, device: str = "cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, std=None, mean=0.0):
        std = shape[-1] ** -0.5 if std is None else std
        return torch.empty(shape, device=device, dtype=BF).normal_(mean, std, generator=g)

    layers = [{
        "attn_norm": normal(HIDDEN, std=0.1, mean=1.0), "qkv": normal((HEADS + 2 * KV_HEADS) * DIM, HIDDEN),
        "o": normal(HIDDEN, HEADS * DIM), "attn_post": normal(HIDDEN, std=0.1, mean=1.0),
        "attn_gate": normal(HIDDEN, std=0.1, mean=1.0), "moe_norm": normal(HIDDEN, std=0.1, mean=1.0),
        "router": normal(EXPERTS, HIDDEN, std=3 * HIDDEN ** -0.5), "gate_up": normal(EXPERTS, 2 * INNER, HIDDEN),
        "down": normal(EXPERTS, HIDDEN, INNER),
    } for _ in range(LAYERS)]
    angle = torch.arange(MAX_POSITION, device=device, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, ROTARY, 2, device=device, dtype=torch.float64) / ROTARY)
    return {"layers": layers, "embedding": normal(VOCAB, HIDDEN, std=1.0), "norm": normal(HIDDEN, std=0.1, mean=1.0),
            "head": normal(VOCAB, HIDDEN), "cos_sin": torch.cat([angle.cos(), angle.sin()], 1).float()}


class Cache:
    """The pages of all layers and each sequence's list of pages."""

    def __init__(self, batch: int, pages: int, device: str = "cuda"):
        shape = (pages, PAGE, KV_HEADS, DIM)
        self.k = [torch.zeros(shape, dtype=BF, device=device) for _ in range(LAYERS)]
        self.v = [torch.zeros(shape, dtype=BF, device=device) for _ in range(LAYERS)]
        self.free = list(range(pages))[::-1]
        self.lengths = [0] * batch
        self.tables = [[] for _ in range(batch)]
        self.device = device

    def extend(self, counts):
        """Room for counts[b] new tokens of each sequence: positions, slots, page table, lengths, starts."""
        positions, slots = [], []
        for b, n in enumerate(counts):
            for p in range(self.lengths[b], self.lengths[b] + n):
                if p % PAGE == 0:
                    self.tables[b].append(self.free.pop())
                positions.append(p)
                slots.append(self.tables[b][p // PAGE] * PAGE + p % PAGE)
            self.lengths[b] += n
        width = max(map(len, self.tables))
        table = [t + [0] * (width - len(t)) for t in self.tables]
        starts = [sum(counts[:b]) for b in range(len(counts) + 1)]
        as_tensor = lambda x, dtype: torch.tensor(x, dtype=dtype, device=self.device)   # noqa: E731
        return (as_tensor(positions, torch.int64), as_tensor(slots, torch.int64), as_tensor(table, torch.int32),
                as_tensor(self.lengths, torch.int32), as_tensor(starts, torch.int32))


def forward(weights, cache, tokens, counts):
    """Logits of the new tokens [sum(counts)] (at most 128 in all)."""
    positions, slots, table, lengths, starts = cache.extend(counts)
    residual = weights["embedding"][tokens].float()            # the residual stream stays in 32 bits
    _, x = residual_norm(residual, pre_weight=weights["layers"][0]["attn_norm"], eps=EPS)
    for i, w in enumerate(weights["layers"]):
        qkv = gemm(x, w["qkv"])
        q, k, v = (z.unflatten(1, (-1, DIM)) for z in qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1))
        q = rope_append(q, k, v, weights["cos_sin"], positions, slots, cache.k[i], cache.v[i])
        o = paged_attention(q, cache.k[i], cache.v[i], table, lengths, starts)
        residual, x = residual_norm(residual, gemm(o.flatten(1), w["o"]), post_weight=w["attn_post"],
                                    gate=w["attn_gate"], pre_weight=w["moe_norm"], eps=EPS)
        following = weights["layers"][i + 1]["attn_norm"] if i + 1 < LAYERS else weights["norm"]
        y = moe(x, w["router"], w["gate_up"], w["down"], TOP_K, scale=BRANCH)
        residual, x = residual_norm(residual, y, pre_weight=following, eps=EPS)
    return gemm(x, weights["head"])


def plain_forward(weights, history, counts):
    """The same logits from the whole token histories in plain torch: 32 bits, rounded where the operators round."""
    def rms(x, w):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()

    out = []
    for seq, n in zip(history, counts):
        t = len(seq)
        residual = weights["embedding"][seq].float()
        half = ROTARY // 2
        cos, sin = weights["cos_sin"][:t, None, :half], weights["cos_sin"][:t, None, half:]

        def turned(z):
            a, b = z.float().split([half, half], -1)
            return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(BF).float()

        x = rms(residual, weights["layers"][0]["attn_norm"]).to(BF)
        for i, w in enumerate(weights["layers"]):
            qkv = (x.float() @ w["qkv"].float().t()).to(BF)
            q, k, v = (z.unflatten(1, (-1, DIM)) for z in qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1))
            q, k, v = turned(q), turned(k).repeat_interleave(HEADS // KV_HEADS, 1), v.float().repeat_interleave(
                HEADS // KV_HEADS, 1)
            s = torch.einsum("ihd,jhd->hij", q, k) * DIM ** -0.5
            s = s.masked_fill(torch.ones(t, t, device=s.device, dtype=torch.bool).triu(1), -float("inf"))
            o = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).to(BF).flatten(1)
            y = (o.float() @ w["o"].float().t()).to(BF).float()
            residual = residual + rms(y, w["attn_post"]) * w["attn_gate"].float()
            x = rms(residual, w["moe_norm"]).to(BF)
            p = (x.float() @ w["router"].float().t()).softmax(-1)
            top, ids = torch.sort(p, dim=-1, descending=True, stable=True)
            top, ids = top[:, :TOP_K], ids[:, :TOP_K]
            top = top / top.sum(-1, keepdim=True) * BRANCH
            gate, up = torch.einsum("th,tkih->tki", x.float(), w["gate_up"].float()[ids]).chunk(2, -1)
            act = (gate * torch.sigmoid(gate) * up).to(BF).float()
            y = torch.einsum("tki,tkhi,tk->th", act, w["down"].float()[ids], top).to(BF)
            residual = residual + y.float()
            following = weights["layers"][i + 1]["attn_norm"] if i + 1 < LAYERS else weights["norm"]
            x = rms(residual, following).to(BF)
        out.append((x[t - n:].float() @ weights["head"].float().t()).to(BF))
    return torch.cat(out)


def generate(prompts, steps: int, seed: int = 0, check: bool = False):
    """Greedy tokens of each prompt; with `check`, also the largest relative error of a step's logits."""
    weights = make_weights(seed)
    cache = Cache(len(prompts), pages=sum((len(p) + steps) // PAGE + 1 for p in prompts))
    history = [list(p) for p in prompts]
    tokens, counts = torch.tensor(sum(prompts, []), device="cuda"), [len(p) for p in prompts]
    worst = 0.0
    for _ in range(steps):
        logits = forward(weights, cache, tokens, counts)
        if check:
            want = plain_forward(weights, [torch.tensor(h, device="cuda") for h in history], counts).float()
            worst = max(worst, float((logits.float() - want).norm() / want.norm()))
        last = torch.tensor(counts, device="cuda").cumsum(0) - 1
        tokens = logits[last].float().argmax(-1)
        for h, t in zip(history, tokens.tolist()):
            h.append(t)
        counts = [1] * len(prompts)
    return [h[len(p):] for h, p in zip(history, prompts)], worst


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, VOCAB, (n,), generator=g).tolist() for n in (37, 1, 64, 19)]
    tokens, worst = generate(prompts, a.steps, check=a.check)
    for p, t in zip(prompts, tokens):
        print("prompt of %2d tokens -> %s" % (len(p), t))
    if a.check:
        print("largest relative error of a step's logits against plain torch: %.2g" % worst)

    # One decode step of the batch, captured in a graph and replayed.
    weights, cache = make_weights(), Cache(len(prompts), pages=64)
    forward(weights, cache, torch.tensor(sum(prompts, []), device="cuda"), [len(p) for p in prompts])
    inputs = cache.extend([1] * len(prompts))
    cache.extend = lambda counts: inputs
    step = torch.zeros(len(prompts), dtype=torch.int64, device="cuda")
    forward(weights, cache, step, [1] * len(prompts))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(weights, cache, step, [1] * len(prompts))
    graph.replay()
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(50):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print("a decode step of %d layers for %d sequences: %.1f us" % (LAYERS, len(prompts), begin.elapsed_time(end) * 20))


if __name__ == "__main__":
    main()
