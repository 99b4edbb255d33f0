"""The decoder-layer operators' C ABI: declarations, exports, workspace sizes and refusals.

CPU-only: every refusal here comes before any device query.
"""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from split_bf16_gemm_swap_gb300 import build, layer, lowm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lowm_layer.h")
PTR = 1 << 20                                          # a 16-byte aligned address that is never read

OK, INVALID, SHAPE, MISALIGNED = (lowm.LOWM_OK, lowm.LOWM_ERR_INVALID_ARGUMENT, lowm.LOWM_ERR_UNSUPPORTED_SHAPE,
                                  lowm.LOWM_ERR_MISALIGNED)


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()
    return lowm.lib()


def declared_functions():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(lowm_\w+)\s*\(", text, flags=re.M)


def test_header_declares_the_binding_functions(library):
    assert tuple(declared_functions()) == layer.ABI_FUNCTIONS
    for name in layer.ABI_FUNCTIONS:
        assert ctypes.cast(getattr(library, name), ctypes.c_void_p).value
        assert layer.function(name)


def test_the_package_exports_the_operators():
    import split_bf16_gemm_swap_gb300 as package
    for name in ("residual_norm", "rope_append", "paged_attention", "moe") + layer.ABI_FUNCTIONS:
        assert callable(getattr(package, name))
    with pytest.raises(AttributeError):
        package.no_such_operator


def test_the_header_is_c99(tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "lowm_layer.h"\nint main(void) { return LOWM_MOE_SOFTMAX; }\n')
    subprocess.check_call([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                           os.path.join(ROOT, "include"), str(src)])


def norm(**kw):
    a = dict(residual=PTR, f32=0, rs=64, block=PTR, bs=64, post=PTR, gate=PTR, gs=0, pre=PTR, out_r=2 * PTR, ors=64,
             out=3 * PTR, os=64, tokens=2, hidden=64, scale=1.0, eps=1e-6, stream=0)
    a.update(kw)
    return layer.lowm_residual_norm(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK), (dict(tokens=0, residual=0, out=0), OK),
    (dict(tokens=-1), INVALID), (dict(hidden=0), INVALID), (dict(hidden=16385), SHAPE),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(residual=0), INVALID), (dict(out=0), INVALID), (dict(out_r=0), INVALID),
    (dict(block=0), INVALID),                          # gate and post weight without a block
    (dict(block=0, post=0, gate=0, out_r=0, scale=0.5), INVALID),
    (dict(os=63), INVALID), (dict(ors=63), INVALID), (dict(rs=-1), INVALID), (dict(bs=-64), INVALID),
    (dict(residual=PTR + 1), MISALIGNED), (dict(f32=1, residual=PTR + 2), MISALIGNED), (dict(out=PTR + 1), MISALIGNED),
    (dict(out=2 * PTR + 128), INVALID),                # out inside out_residual
])
def test_norm_refusals(kw, want):
    assert norm(**kw) == want


@pytest.mark.parametrize("kw", [
    dict(out=2 * PTR + 64, ors=128, os=128), dict(out=2 * PTR - 64, ors=128, os=128),
    dict(out=2 * PTR + 256, ors=128, os=128), dict(out=2 * PTR - 256, ors=128, os=128),
    dict(out=2 * PTR + 128, f32=1, ors=96, os=192), dict(out=2 * PTR + 128, ors=128, os=136),
])
def test_norm_refuses_outputs_that_share_rows(kw):
    assert norm(**kw) == INVALID


def rope(**kw):
    a = dict(q=PTR, qt=256, qh=64, k=PTR, kt=256, kh=64, v=PTR, vt=256, vh=64, table=PTR, rows=100, pos=PTR, ps=0,
             axes=1, s0=32, s1=0, inter=0, slots=PTR, out=PTR, ot=256, oh=64, kc=PTR, kp=4096, kl=256, kch=64,
             vc=PTR, vp=4096, vl=256, vch=64, pages=4, page=16, tokens=2, heads=4, kv_heads=4, dim=64, rotary=64,
             stream=0)
    a.update(kw)
    return layer.lowm_rope_append(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK), (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(axes=0), INVALID), (dict(axes=4), INVALID), (dict(page=0), INVALID), (dict(dim=1025), SHAPE),
    (dict(rotary=66), SHAPE), (dict(rotary=63), SHAPE), (dict(s0=31), INVALID), (dict(s0=33), INVALID),
    (dict(axes=2, s0=16, s1=15), INVALID), (dict(axes=3, s0=16, s1=17), INVALID),
    (dict(q=0), INVALID), (dict(table=0), INVALID), (dict(pos=0), INVALID), (dict(slots=0), INVALID),
    (dict(kc=0), INVALID), (dict(vp=-1), INVALID), (dict(q=PTR + 1), MISALIGNED), (dict(table=PTR + 4), MISALIGNED),
    (dict(slots=PTR + 4), MISALIGNED),
])
def test_rope_refusals(kw, want):
    assert rope(**kw) == want


def attention(**kw):
    a = dict(q=PTR, qt=256, qh=64, kc=PTR, kp=4096, kl=256, kch=64, vc=PTR, vp=4096, vl=256, vch=64, pages=4, page=16,
             table=PTR, ts=4, width=4, lens=PTR, cu=PTR, out=PTR, ot=256, oh=64, lse=0, batch=2, q_tokens=2, heads=4,
             kv_heads=4, dim=64, scale=0.1, window=0, work=PTR, nbytes=1 << 40, stream=0)
    a.update(kw)
    return layer.lowm_paged_attention(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q_tokens=0), OK), (dict(q_tokens=-1), INVALID), (dict(batch=-1), INVALID), (dict(heads=0), INVALID),
    (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(width=-1), INVALID),
    (dict(dim=96), SHAPE), (dict(page=12), SHAPE), (dict(page=4), SHAPE), (dict(page=2048), SHAPE),
    (dict(heads=6), SHAPE), (dict(heads=516), SHAPE),
    (dict(q=0), INVALID), (dict(kc=0), INVALID), (dict(table=0), INVALID), (dict(cu=0), INVALID),
    (dict(work=0), INVALID), (dict(nbytes=0), INVALID), (dict(kp=-8), INVALID), (dict(qt=-1), INVALID),
    (dict(kl=260), MISALIGNED), (dict(kc=PTR + 8), MISALIGNED), (dict(work=PTR + 8), MISALIGNED),
    (dict(out=PTR + 1), MISALIGNED), (dict(lens=PTR + 2), MISALIGNED),
])
def test_attention_refusals(kw, want):
    assert attention(**kw) == want


def test_attention_refuses_a_line_of_tiles_past_32_bits():
    # 128 (2^24 - 1) places: 2^31 - 128, which rounding up to equal shares takes past 2^31
    assert attention(batch=128, q_tokens=1, heads=1, kv_heads=1, width=16777205, ts=16777205, page=64) == SHAPE


def moe(**kw):
    a = dict(x=PTR, xs=64, router=PTR, bias=0, gate_up=PTR, down=PTR, out=PTR, os=64, tokens=2, hidden=64, inner=32,
             experts=8, top_k=2, scoring=0, renorm=1, scale=1.0, work=PTR, nbytes=1 << 40, stream=0)
    a.update(kw)
    return layer.lowm_moe(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK), (dict(tokens=-1), INVALID), (dict(tokens=129), SHAPE), (dict(hidden=60), SHAPE),
    (dict(inner=36), SHAPE), (dict(experts=1025), SHAPE), (dict(top_k=17, experts=32), SHAPE),
    (dict(top_k=9), INVALID), (dict(top_k=0), INVALID), (dict(scoring=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(x=0), INVALID), (dict(router=0), INVALID), (dict(work=0), INVALID), (dict(nbytes=8), INVALID),
    (dict(os=63), INVALID), (dict(xs=-64), INVALID), (dict(xs=68), MISALIGNED), (dict(x=PTR + 2), MISALIGNED),
    (dict(down=PTR + 8), MISALIGNED), (dict(bias=PTR + 2), MISALIGNED), (dict(out=PTR + 1), MISALIGNED),
])
def test_moe_refusals(kw, want):
    assert moe(**kw) == want


def test_workspace_sizes():
    assert layer.lowm_paged_attention_workspace(4, 4, 32, 8, 128) > 0
    assert layer.lowm_paged_attention_workspace(0, 0, 32, 8, 64) > 0
    for bad in ((4, 4, 32, 8, 96), (4, 4, 30, 8, 128), (-1, 4, 32, 8, 128), (4, 4, 0, 8, 128), (4, 4, 2048, 8, 128)):
        assert layer.lowm_paged_attention_workspace(*bad) == 0
    assert layer.lowm_moe_workspace(128, 4096, 1400, 32, 4) > 0
    for bad in ((129, 64, 32, 8, 2), (2, 60, 32, 8, 2), (2, 64, 32, 8, 9), (2, 64, 32, 2000, 2), (2, 64, 0, 8, 2)):
        assert layer.lowm_moe_workspace(*bad) == 0


def test_python_refusals_need_no_gpu():
    import torch
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        layer.residual_norm(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        layer.moe(x, x, x, x, 1)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        layer.paged_attention(q, q, q, q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        layer.rope_append(q, q, q, q, q, q, q, q)
