"""The C ABI of the 8-bit operators and of the pages: declarations, exports, workspace sizes and refusals.

CPU-only: every refusal here comes before any device query.
"""
from __future__ import annotations

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from split_bf16_gemm_swap_gb300 import build, fp8, layer, lowm, pages

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PTR = 1 << 20                                          # a 16-byte aligned address that is never read

OK, INVALID, SHAPE, MISALIGNED = (lowm.LOWM_OK, lowm.LOWM_ERR_INVALID_ARGUMENT, lowm.LOWM_ERR_UNSUPPORTED_SHAPE,
                                  lowm.LOWM_ERR_MISALIGNED)


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()
    return lowm.lib()


@pytest.mark.parametrize("header,module", [("lowm_fp8.h", fp8), ("lowm_pages.h", pages)])
def test_header_declares_the_binding_functions(library, header, module):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    declared = re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(lowm_\w+)\s*\(", text, flags=re.M)
    assert tuple(declared) == module.ABI_FUNCTIONS
    import split_bf16_gemm_swap_gb300 as package
    for name in module.ABI_FUNCTIONS:
        assert ctypes.cast(getattr(library, name), ctypes.c_void_p).value
        assert layer.function(name)
        assert callable(getattr(package, name))


def test_the_package_exports_the_operators():
    import split_bf16_gemm_swap_gb300 as package
    for name in ("quantize_fp8", "gemm_fp8", "rope_append_fp8", "paged_attention_fp8", "fork_pages", "extend_pages",
                 "compact_pages", "copy_pages"):
        assert callable(getattr(package, name))


def test_the_headers_are_c99(tmp_path):
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "lowm_fp8.h"\n#include "lowm_pages.h"\nint main(void) { lowm_page_span_t s = {0, 0, 0}; return (int)s.page_bytes; }\n')
    subprocess.check_call([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                           os.path.join(ROOT, "include"), str(src)])


def test_the_page_span_lies_as_the_binding_packs_it():
    assert ctypes.sizeof(pages.lowm_page_span_t) == 24
    assert [getattr(pages.lowm_page_span_t, n).offset for n in ("base", "page_stride", "page_bytes")] == [0, 8, 16]


# -------------------------------------------------------------------------------------------- products
def quantize(**kw):
    a = dict(x=PTR, xs=64, codes=PTR, scales=PTR, rows=2, cols=64, block=1, stream=0)
    a.update(kw)
    return fp8.lowm_quantize_fp8(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), OK), (dict(rows=0, x=0, codes=0, scales=0), OK), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(block=2), INVALID), (dict(block=0), INVALID), (dict(xs=-1), INVALID), (dict(x=0), INVALID), (dict(codes=0), INVALID),
    (dict(scales=0), INVALID), (dict(x=PTR + 1), MISALIGNED), (dict(scales=PTR + 2), MISALIGNED),
    (dict(rows=2 ** 31 - 1, cols=2 ** 31 - 1), SHAPE),
])
def test_quantize_refusals(kw, want):
    assert quantize(**kw) == want


def gemm(**kw):
    a = dict(A=PTR, sa=PTR, W=PTR, sw=PTR, C=PTR, M=4, N=128, K=128, flags=0, stream=0)
    a.update(kw)
    return fp8.lowm_gemm_fp8(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), INVALID), (dict(M=-1), INVALID), (dict(M=129), SHAPE), (dict(N=0), INVALID), (dict(K=0), INVALID),
    (dict(K=24), SHAPE), (dict(N=(1 << 30) + 1), SHAPE), (dict(flags=2), INVALID), (dict(flags=4), INVALID), (dict(A=0), INVALID),
    (dict(sa=0), INVALID), (dict(W=0), INVALID), (dict(sw=0), INVALID), (dict(C=0), INVALID), (dict(A=PTR + 8), MISALIGNED),
    (dict(W=PTR + 8), MISALIGNED), (dict(C=PTR + 1), MISALIGNED), (dict(sa=PTR + 2), MISALIGNED), (dict(sw=PTR + 1), MISALIGNED),
])
def test_gemm_refusals(kw, want):
    assert gemm(**kw) == want


def gemm_bf16(**kw):
    a = dict(x=PTR, xs=128, W=PTR, sw=PTR, C=PTR, M=4, N=128, K=128, flags=0, work=PTR, nbytes=1 << 30, stream=0)
    a.update(kw)
    return fp8.lowm_gemm_fp8_bf16(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(M=0), INVALID), (dict(M=129), SHAPE), (dict(K=8), SHAPE), (dict(flags=8), INVALID), (dict(x=0), INVALID),
    (dict(W=0), INVALID), (dict(sw=0), INVALID), (dict(C=0), INVALID), (dict(xs=-128), INVALID), (dict(work=0), INVALID),
    (dict(nbytes=0), INVALID), (dict(M=100, nbytes=100 * 128), INVALID), (dict(x=PTR + 1), MISALIGNED),
    (dict(work=PTR + 8), MISALIGNED), (dict(W=PTR + 4), MISALIGNED),
])
def test_gemm_of_bf16_refusals(kw, want):
    assert gemm_bf16(**kw) == want


# ------------------------------------------------------------------------------------------- the cache
def rope(**kw):
    a = dict(q=PTR, qt=256, qh=64, k=PTR, kt=256, kh=64, v=PTR, vt=256, vh=64, table=PTR, rows=100, pos=PTR, ps=0,
             axes=1, s0=32, s1=0, inter=0, slots=PTR, out=PTR, ot=256, oh=64, kc=PTR, kp=4096, kl=256, kch=64,
             vc=PTR, vp=4096, vl=256, vch=64, ks=PTR, ksp=8, ksb=4, ksh=1, vs=PTR, vsp=8, vsb=4, vsh=1, pages=4, page=16, block=8,
             tokens=2, heads=4, kv_heads=4, dim=64, rotary=64, stream=0)
    a.update(kw)
    return fp8.lowm_rope_append_fp8(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=0), OK), (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(axes=0), INVALID), (dict(axes=4), INVALID), (dict(page=0), INVALID), (dict(block=0), INVALID), (dict(block=3), SHAPE),
    (dict(block=32), SHAPE), (dict(dim=257), SHAPE), (dict(rotary=66), SHAPE), (dict(rotary=63), SHAPE), (dict(s0=31), INVALID),
    (dict(axes=2, s0=16, s1=15), INVALID), (dict(axes=3, s0=16, s1=17), INVALID), (dict(q=0), INVALID), (dict(table=0), INVALID),
    (dict(slots=0), INVALID), (dict(kc=0), INVALID), (dict(ks=0), INVALID), (dict(vs=0), INVALID), (dict(vp=-1), INVALID),
    (dict(ksb=-4), INVALID), (dict(q=PTR + 1), MISALIGNED), (dict(table=PTR + 4), MISALIGNED), (dict(slots=PTR + 4), MISALIGNED),
    (dict(vs=PTR + 1), MISALIGNED), (dict(tokens=2 ** 31 - 1, heads=1000), SHAPE),
])
def test_rope_refusals(kw, want):
    assert rope(**kw) == want


def attention(**kw):
    a = dict(q=PTR, qt=256, qh=64, kc=PTR, kp=4096, kl=256, kch=64, vc=PTR, vp=4096, vl=256, vch=64, ks=PTR, ksp=8, ksb=4, ksh=1,
             vs=PTR, vsp=8, vsb=4, vsh=1, pages=4, page=16, block=8, table=PTR, ts=4, width=4, lens=PTR, cu=PTR, out=PTR, ot=256,
             oh=64, lse=0, batch=2, q_tokens=2, heads=4, kv_heads=4, dim=64, scale=0.1, window=0, work=PTR, nbytes=1 << 40, stream=0)
    a.update(kw)
    return fp8.lowm_paged_attention_fp8(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(q_tokens=0), OK), (dict(q_tokens=-1), INVALID), (dict(batch=-1), INVALID), (dict(heads=0), INVALID),
    (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(width=-1), INVALID), (dict(block=0), INVALID),
    (dict(block=32), SHAPE), (dict(block=6), SHAPE), (dict(dim=96), SHAPE), (dict(page=12), SHAPE), (dict(page=4, block=4), SHAPE),
    (dict(page=2048), SHAPE), (dict(heads=6), SHAPE), (dict(heads=516), SHAPE), (dict(q=0), INVALID), (dict(kc=0), INVALID),
    (dict(ks=0), INVALID), (dict(vs=0), INVALID), (dict(table=0), INVALID), (dict(cu=0), INVALID), (dict(work=0), INVALID),
    (dict(nbytes=0), INVALID), (dict(kp=-16), INVALID), (dict(qt=-1), INVALID), (dict(ksp=-1), INVALID), (dict(kl=264), MISALIGNED),
    (dict(kc=PTR + 8), MISALIGNED), (dict(work=PTR + 8), MISALIGNED), (dict(out=PTR + 1), MISALIGNED), (dict(ks=PTR + 1), MISALIGNED),
    (dict(lens=PTR + 2), MISALIGNED),
])
def test_attention_refusals(kw, want):
    assert attention(**kw) == want


def test_attention_refuses_a_line_of_tiles_past_32_bits():
    assert attention(batch=128, q_tokens=1, heads=1, kv_heads=1, width=16777205, ts=16777205, page=64) == SHAPE


def test_workspace_sizes():
    few = fp8.lowm_paged_attention_fp8_workspace(4, 4, 32, 8, 128, 64, 100)
    assert 0 < few == fp8.lowm_paged_attention_fp8_workspace(4, 4, 32, 8, 128, 64, 100000)
    # many rows a sequence: the widened keys and values of 6400 tokens, and more
    many = fp8.lowm_paged_attention_fp8_workspace(1, 500, 32, 8, 128, 64, 100)
    assert many > 2 * 6400 * 8 * 128 * 2
    # where they would pass the limit the cache is read as it is
    assert fp8.lowm_paged_attention_fp8_workspace(1, 500, 32, 8, 128, 64, 1 << 20) < 1 << 30
    for bad in ((4, 4, 32, 8, 96, 64, 4), (4, 4, 30, 8, 128, 64, 4), (-1, 4, 32, 8, 128, 64, 4), (4, 4, 32, 8, 128, 0, 4),
                (4, 4, 2048, 8, 128, 64, 4), (4, 4, 32, 8, 128, 64, -1)):
        assert fp8.lowm_paged_attention_fp8_workspace(*bad) == 0
    assert fp8.lowm_gemm_fp8_bf16_workspace(16, 4096) > 0
    assert fp8.lowm_gemm_fp8_bf16_workspace(128, 4096) >= 128 * 4096 + 128 * 32 * 4
    for bad in ((0, 4096), (129, 4096), (4, 0), (4, 40)):
        assert fp8.lowm_gemm_fp8_bf16_workspace(*bad) == 0
    assert pages.lowm_extend_pages_workspace(100) >= 400 and pages.lowm_extend_pages_workspace(0) == 0
    assert pages.lowm_compact_pages_workspace(5000) >= 5000 * 4 + 8 and pages.lowm_compact_pages_workspace(-1) == 0


@pytest.mark.parametrize("batch,width", [(8, 2048), (17, 2048), (64, 2048), (3, 16384), (1000, 64)])
def test_the_attention_workspace_is_bounded(batch, width):
    # copies of 1 to 16 GiB in all; never more than one at a time, and every call is still widened
    size = lambda w: fp8.lowm_paged_attention_fp8_workspace(batch, 30 * batch, 32, 8, 128, 64, w)   # noqa: E731
    assert size(0) < 1 << 26 and 1 << 29 < size(width) < (1 << 30) + (1 << 26)


# ----------------------------------------------------------------------------------------------- pages
def fork(**kw):
    a = dict(table=PTR, ts=4, lens=PTR, rows=2, parents=PTR, new_rows=2, width=4, refs=PTR, pages=8, page=16, out=2 * PTR, os=4,
             new_lens=PTR, src=PTR, dst=PTR, missing=PTR, stream=0)
    a.update(kw)
    return pages.lowm_fork_pages(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(new_rows=-1), INVALID), (dict(width=-1), INVALID), (dict(pages=0), INVALID),
    (dict(page=0), INVALID), (dict(table=0), INVALID), (dict(out=0), INVALID), (dict(lens=0), INVALID), (dict(parents=0), INVALID),
    (dict(refs=0), INVALID), (dict(src=0), INVALID), (dict(dst=0), INVALID), (dict(missing=0), INVALID), (dict(ts=3), INVALID),
    (dict(os=3), INVALID), (dict(out=PTR), INVALID), (dict(rows=8193), SHAPE), (dict(new_rows=8193), SHAPE),
    (dict(table=PTR + 2), MISALIGNED), (dict(refs=PTR + 1), MISALIGNED),
])
def test_fork_refusals(kw, want):
    assert fork(**kw) == want



@pytest.mark.parametrize("kw", [
    dict(out=PTR + 16), dict(out=PTR - 16), dict(out=PTR + 4), dict(ts=8, os=8, out=PTR + 12), dict(ts=8, os=8, out=PTR - 12),
    dict(ts=8, os=8, out=PTR + 32 + 12), dict(ts=8, os=4, out=PTR + 32), dict(ts=10, os=10, out=PTR + 28, width=5),
])
def test_fork_refuses_a_new_table_that_meets_the_old_one(kw):
    assert fork(**kw) == INVALID


def extend(**kw):
    a = dict(table=PTR, ts=4, lens=PTR, rows=2, width=4, cu=PTR, tokens=3, refs=PTR, pages=8, page=16, pos=PTR, slots=PTR,
             missing=PTR, work=PTR, nbytes=1 << 20, stream=0)
    a.update(kw)
    return pages.lowm_extend_pages(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(tokens=-1), INVALID), (dict(pages=0), INVALID), (dict(page=-1), INVALID), (dict(cu=0), INVALID),
    (dict(pos=0), INVALID), (dict(slots=0), INVALID), (dict(missing=0), INVALID), (dict(work=0), INVALID), (dict(nbytes=31), INVALID),
    (dict(ts=2), INVALID), (dict(rows=8193, ts=8), SHAPE), (dict(slots=PTR + 4), MISALIGNED), (dict(lens=PTR + 2), MISALIGNED),
])
def test_extend_refusals(kw, want):
    assert extend(**kw) == want


def compact(**kw):
    a = dict(table=PTR, ts=4, lens=PTR, rows=2, width=4, refs=PTR, pages=8, page=16, src=PTR, dst=PTR, used=PTR, work=PTR,
             nbytes=1 << 20, stream=0)
    a.update(kw)
    return pages.lowm_compact_pages(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(refs=0), INVALID), (dict(src=0), INVALID),
    (dict(dst=0), INVALID), (dict(used=0), INVALID), (dict(work=0), INVALID), (dict(nbytes=35), INVALID), (dict(lens=0), INVALID),
    (dict(dst=PTR + 2), MISALIGNED),
])
def test_compact_refusals(kw, want):
    assert compact(**kw) == want


def copy(spans=((PTR, 64, 64),), src=PTR, dst=PTR, pairs=2, num_pages=8):
    packed = (pages.lowm_page_span_t * len(spans))(*spans)
    return pages.lowm_copy_pages(packed if spans else None, len(spans), src, dst, pairs, num_pages, 0)


@pytest.mark.parametrize("kw,want", [
    (dict(spans=()), OK), (dict(pairs=0, src=0, dst=0), OK), (dict(num_pages=0), OK), (dict(pairs=-1), INVALID),
    (dict(num_pages=-1), INVALID), (dict(src=0), INVALID), (dict(dst=0), INVALID), (dict(spans=((PTR, 63, 64),)), INVALID),
    (dict(spans=((0, 64, 64),)), INVALID), (dict(spans=((PTR, -64, 64),)), INVALID), (dict(spans=((PTR, 64, -1),)), INVALID),
    (dict(src=PTR + 2), MISALIGNED),
])
def test_copy_refusals(kw, want):
    assert copy(**kw) == want


# ---------------------------------------------------------------------------------------------- Python
def test_python_refusals_need_no_gpu():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 4, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: fp8.quantize_fp8(x), lambda: fp8.gemm_fp8(x, x, x), lambda: fp8.rope_append_fp8(q, q, q, *[x] * 7),
                 lambda: fp8.paged_attention_fp8(q, *[x] * 7), lambda: pages.fork_pages(i, i, i, i, 16),
                 lambda: pages.extend_pages(i, i, i, i, 16, 1), lambda: pages.compact_pages(i, i, i, 16),
                 lambda: pages.copy_pages([x], i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
