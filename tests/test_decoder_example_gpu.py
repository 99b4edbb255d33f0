"""The example decoder: GEMM, norms, rotary append, paged attention and experts together against plain torch."""
from __future__ import annotations

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decoder_layer
        yield decoder_layer
    finally:
        sys.path.pop(0)


def test_generation_matches_plain_torch(example):
    prompts = [[5, 9, 200, 7] * 9, [3], list(range(50)), [1000] * 17]
    tokens, worst = example.generate(prompts, 6, check=True)
    assert [len(t) for t in tokens] == [6] * 4
    # Both sides round to bf16 at the same places (the plain one not the attention weights); what differs is a
    # rounding here and there, 2^-9 of a value, through three layers of five roundings.
    assert worst < 15 * 2.0 ** -9


def test_ragged_batch_gives_each_sequence_its_own_tokens(example):
    a, b = list(range(40, 73)), [7, 8]
    together, _ = example.generate([a, b], 4)
    assert together == [example.generate([a], 4)[0][0], example.generate([b], 4)[0][0]]
