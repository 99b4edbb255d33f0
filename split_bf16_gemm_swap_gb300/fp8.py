"""ctypes binding of the 8-bit operators in ``include/lowm_fp8.h``.

:func:`quantize_fp8`, :func:`gemm_fp8`, :func:`rope_append_fp8` and
:func:`paged_attention_fp8` take torch tensors, check them, make the outputs
that are not given and launch, in the manner of :mod:`.layer` (streams, devices,
workspaces and errors are described there).  Codes are ``torch.float8_e4m3fn``,
scales fp32.  There is no fallback.  Inference only.
"""
from __future__ import annotations

import functools
import math

import torch

from . import layer
from .layer import _cuda, _current_device, _current_stream, _dense, _f, _i, _launch, _on, _p, _row_stride, _rows, _z, function
from .lowm import LOWM_OK, LowmError

# Exported C functions, in header order.
ABI_FUNCTIONS = (
    "lowm_quantize_fp8",
    "lowm_gemm_fp8",
    "lowm_gemm_fp8_bf16",
    "lowm_gemm_fp8_bf16_workspace",
    "lowm_rope_append_fp8",
    "lowm_paged_attention_fp8",
    "lowm_paged_attention_fp8_workspace",
)

# 64-bit strides and counts: a pointer's integer takes ctypes 0.02 us on the host, a c_int64's 0.06, and the append has 26.
_s = _p
_cache = [_p, _s, _s, _s]                  # a pointer and three strides
layer._ARGTYPES.update({
    "lowm_quantize_fp8": [_p, _s, _p, _p, _i, _i, _i, _p],
    "lowm_gemm_fp8": [_p, _p, _p, _p, _p, _i, _i, _i, _i, _p],
    "lowm_gemm_fp8_bf16": [_p, _s, _p, _p, _p, _i, _i, _i, _i, _p, _z, _p],
    "lowm_gemm_fp8_bf16_workspace": [_i, _i],
    "lowm_rope_append_fp8": [_p, _s, _s, _p, _s, _s, _p, _s, _s, _p, _s, _p, _s, _i, _i, _i, _i, _p, _p, _s, _s,
                             *_cache, *_cache, *_cache, *_cache, _s, _i, _i, _i, _i, _i, _i, _i, _p],
    "lowm_paged_attention_fp8": [_p, _s, _s, *_cache, *_cache, *_cache, *_cache, _s, _i, _i, _p, _s, _i, _p, _p, _p, _s, _s,
                                 _p, _i, _i, _i, _i, _i, _f, _i, _p, _z, _p],
    "lowm_paged_attention_fp8_workspace": [_i] * 7,
})

FP8 = torch.float8_e4m3fn
BLOCK = 128                                # columns of a scale of quantize_fp8 and gemm_fp8


def lowm_quantize_fp8(*args) -> int:
    return function("lowm_quantize_fp8")(*args)


def lowm_gemm_fp8(*args) -> int:
    return function("lowm_gemm_fp8")(*args)


def lowm_gemm_fp8_bf16(*args) -> int:
    return function("lowm_gemm_fp8_bf16")(*args)


def lowm_gemm_fp8_bf16_workspace(M: int, K: int) -> int:
    return function("lowm_gemm_fp8_bf16_workspace")(M, K)


def lowm_rope_append_fp8(*args) -> int:
    return function("lowm_rope_append_fp8")(*args)


def lowm_paged_attention_fp8(*args) -> int:
    return function("lowm_paged_attention_fp8")(*args)


def lowm_paged_attention_fp8_workspace(batch: int, q_tokens: int, heads: int, kv_heads: int, dim: int, page_size: int,
                                       table_width: int) -> int:
    return function("lowm_paged_attention_fp8_workspace")(batch, q_tokens, heads, kv_heads, dim, page_size, table_width)


_gemm_bytes = functools.lru_cache(maxsize=4096)(lowm_gemm_fp8_bf16_workspace)
_attention_bytes = functools.lru_cache(maxsize=4096)(lowm_paged_attention_fp8_workspace)


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def quantize_fp8(x, block_rows: int = 1, *, out=None, out_scale=None, stream=None):
    """Codes and scales of a bf16 matrix: ``(codes, scales)`` with x about codes * scale.

    x [rows, cols] bf16; a scale stands for `block_rows` rows (1: activations,
    128: weights) and 128 columns.  codes [rows, cols] float8_e4m3fn, scales
    [ceil(rows / block_rows), ceil(cols / 128)] fp32, powers of two.
    """
    device = _cuda(x, "x")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return quantize_fp8(x, block_rows, out=out, out_scale=out_scale)
    if x.dim() != 2:
        raise ValueError("x must be [rows, cols]")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    shape = x.shape
    rows, cols = shape
    scale_shape = (-(-rows // block_rows), _blocks(cols))
    stride = _row_stride(x, "x", torch.bfloat16, shape, device)
    if out is None:
        out = torch.empty(shape, dtype=FP8, device=x.device)
    else:
        _dense(out, "out", FP8, shape, device)
    if out_scale is None:
        out_scale = torch.empty(scale_shape, dtype=torch.float32, device=x.device)
    else:
        _dense(out_scale, "out_scale", torch.float32, scale_shape, device)
    s = function("lowm_quantize_fp8")(x.data_ptr(), stride, out.data_ptr(), out_scale.data_ptr(), rows, cols, block_rows,
                                      _current_stream(device))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_quantize_fp8")
    return out, out_scale


def gemm_fp8(A, W, W_scale, A_scale=None, *, out=None, flags: int = 0, stream=None):
    """C = A . W^T in 8 bits with scales by block of 128; C bf16 [M, N], M at most 128.

    W [N, K] float8_e4m3fn with W_scale [ceil(N / 128), ceil(K / 128)] fp32 (of
    ``quantize_fp8(w, 128)`` or a checkpoint); A [M, K] float8_e4m3fn with A_scale
    [M, ceil(K / 128)] (of ``quantize_fp8(x)``), or bf16 without one: it is
    quantised within the call.  K a multiple of 16.  flags:
    LOWM_FLAG_W_BEFORE_PDL_WAIT when the kernel before this call on the stream does
    not write W.
    """
    device = _cuda(A, "A")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return gemm_fp8(A, W, W_scale, A_scale, out=out, flags=flags)
    if A.dim() != 2 or W.dim() != 2 or A.shape[1] != W.shape[1]:
        raise ValueError("A must be [M, K] and W [N, K]")
    shape = A.shape
    M, K = shape
    N = W.shape[0]
    blocks = _blocks(K)
    _dense(W, "W", FP8, (N, K), device)
    _dense(W_scale, "W_scale", torch.float32, (_blocks(N), blocks), device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    else:
        _dense(out, "out", torch.bfloat16, (M, N), device)
    if A_scale is not None:
        _dense(A, "A", FP8, shape, device)
        _dense(A_scale, "A_scale", torch.float32, (M, blocks), device)
        s = function("lowm_gemm_fp8")(A.data_ptr(), A_scale.data_ptr(), W.data_ptr(), W_scale.data_ptr(), out.data_ptr(), M, N,
                                      K, flags, _current_stream(device))
        if s != LOWM_OK:
            raise LowmError(s, "lowm_gemm_fp8")
        return out
    stride = _row_stride(A, "A", torch.bfloat16, shape, device)
    _launch("lowm_gemm_fp8_bf16", (A.data_ptr(), stride, W.data_ptr(), W_scale.data_ptr(), out.data_ptr(), M, N, K, flags),
            _gemm_bytes(M, K), device, _current_stream(device))
    return out


def _codes(k_cache, v_cache, k_scale, v_scale, device: int):
    """Checks of a cache of codes; its arguments for the library, from the pointer of k_cache to the block."""
    shape, scale_shape, f32 = k_cache.shape, k_scale.shape, torch.float32
    if len(shape) != 4 or len(scale_shape) != 3:
        raise ValueError("the caches must be [num_pages, page_size, kv_heads, dim] and the scales [num_pages, page_size / block, "
                         "kv_heads]")
    num_pages, page_size, kv_heads, dim = shape
    scale_pages, blocks, scale_heads = scale_shape
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if (k_cache.dtype is not FP8 or v_cache.dtype is not FP8 or k_scale.dtype is not f32 or v_scale.dtype is not f32
            or v_cache.shape != shape or v_scale.shape != scale_shape or scale_pages != num_pages or scale_heads != kv_heads
            or blocks < 1 or page_size % blocks or (dim > 1 and (k3 != 1 or v3 != 1)) or k_cache.get_device() != device
            or v_cache.get_device() != device or k_scale.get_device() != device or v_scale.get_device() != device):
        _refuse_codes(k_cache, v_cache, k_scale, v_scale, device)
    return (k_cache.data_ptr(), k0, k1, k2, v_cache.data_ptr(), v0, v1, v2, k_scale.data_ptr(), *k_scale.stride(),
            v_scale.data_ptr(), *v_scale.stride(), num_pages, page_size, page_size // blocks)


def _refuse_codes(k_cache, v_cache, k_scale, v_scale, device: int):
    num_pages, page_size, kv_heads, _ = k_cache.shape
    blocks = k_scale.shape[1]
    _rows(k_cache, "k_cache", FP8, k_cache.shape, device)
    _rows(v_cache, "v_cache", FP8, k_cache.shape, device)
    if blocks < 1 or page_size % blocks:
        raise ValueError("page_size %d is not a whole number of %d blocks" % (page_size, blocks))
    for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
        if x.dtype is not torch.float32 or x.shape != (num_pages, blocks, kv_heads) or x.get_device() != device:
            layer._refuse(x, name, torch.float32, torch.Size((num_pages, blocks, kv_heads)), device)
    raise AssertionError("unreachable")


def rope_append_fp8(q, k, v, cos_sin, positions, slots, k_cache, v_cache, k_scale, v_scale, *, sections=None,
                    interleaved: bool = False, out=None, stream=None):
    """:func:`.layer.rope_append` into a cache of codes with a scale by block of tokens and head; returns the rotated q.

    k_cache, v_cache [num_pages, page_size, kv_heads, dim] float8_e4m3fn; k_scale,
    v_scale [num_pages, page_size / block, kv_heads] fp32.  Tokens that share a
    block are to be neighbours with rising slots.  Where they begin inside a block,
    the tokens before them stay, their codes moved to a larger scale if the new
    ones need it; where they begin a block, it begins anew.
    """
    device = _cuda(q, "q")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return rope_append_fp8(q, k, v, cos_sin, positions, slots, k_cache, v_cache, k_scale, v_scale, sections=sections,
                                   interleaved=interleaved, out=out)
    bf16, i64 = torch.bfloat16, torch.int64
    if q.dim() != 3 or k.dim() != 3 or cos_sin.dim() != 2:
        raise ValueError("q and k must be [tokens, heads, dim] and cos_sin [table_rows, rotary]")
    q_shape = q.shape
    tokens, heads, dim = q_shape
    kv_heads = k.shape[1]
    table_shape = cos_sin.shape
    table_rows, rotary = table_shape
    kv_shape = (tokens, kv_heads, dim)
    qs = _rows(q, "q", bf16, q_shape, device)
    ks = _rows(k, "k", bf16, kv_shape, device)
    vs = _rows(v, "v", bf16, kv_shape, device)
    _dense(cos_sin, "cos_sin", torch.float32, table_shape, device)
    _dense(slots, "slots", i64, (tokens,), device)
    cache = _codes(k_cache, v_cache, k_scale, v_scale, device)
    if k_cache.shape[2:] != (kv_heads, dim):
        raise ValueError("the caches' heads and head size must be those of k, %d and %d" % (kv_heads, dim))
    axes, positions_stride, section0, section1 = _axes(positions, sections, tokens, rotary, device)
    if out is None:
        out = torch.empty(q_shape, dtype=bf16, device=q.device)
    os = _rows(out, "out", bf16, q_shape, device)
    s = function("lowm_rope_append_fp8")(
        q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], cos_sin.data_ptr(), table_rows,
        positions.data_ptr(), positions_stride, axes, section0, section1, interleaved, slots.data_ptr(), out.data_ptr(), os[0],
        os[1], *cache, tokens, heads, kv_heads, dim, rotary, _current_stream(device))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_rope_append_fp8")
    return out


def _axes(positions, sections, tokens: int, rotary: int, device: int):
    if positions.dim() == 1:
        _dense(positions, "positions", torch.int64, (tokens,), device)
        if sections is not None and tuple(sections) != (rotary // 2,):
            raise ValueError("sections of one axis must be (rotary / 2,)")
        return 1, 0, rotary // 2, 0
    axes = positions.shape[0]
    stride = _rows(positions, "positions", torch.int64, (axes, tokens), device)[0]
    if sections is None or not 1 <= axes <= 3 or len(sections) != axes or sum(sections) * 2 != rotary:
        raise ValueError("positions [axes, tokens] need one to three axes and a section (rotary pairs) of each, "
                         "rotary / 2 in all")
    return axes, stride, sections[0], sections[1] if axes > 1 else 0


def paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, cu_q, *, scale=None, window: int = 0,
                        out=None, return_lse: bool = False, stream=None):
    """:func:`.layer.paged_attention` over a cache of codes with their scales, as :func:`rope_append_fp8` keeps it.

    q and the result are bf16; k_cache, v_cache float8_e4m3fn; k_scale, v_scale
    [num_pages, page_size / block, kv_heads] fp32.  v_scale is from 0 to 2^50 (less
    than 2^-50 counts as 2^-50); another one makes the rows that see its tokens NaN.
    """
    device = _cuda(q, "q")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return paged_attention_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, kv_lens, cu_q, scale=scale,
                                       window=window, out=out, return_lse=return_lse)
    bf16, i32 = torch.bfloat16, torch.int32
    if q.dim() != 3 or page_table.dim() != 2:
        raise ValueError("q must be [q_tokens, heads, dim] and page_table [batch, table_width]")
    q_shape, table_shape = q.shape, page_table.shape
    q_tokens, heads, dim = q_shape
    batch, table_width = table_shape
    cache = _codes(k_cache, v_cache, k_scale, v_scale, device)
    kv_heads = k_cache.shape[2]
    if k_cache.shape[3] != dim:
        raise ValueError("q and the caches must have one head size, not %d and %d" % (dim, k_cache.shape[3]))
    qs = _rows(q, "q", bf16, q_shape, device)
    table_stride = _rows(page_table, "page_table", i32, table_shape, device)[0]
    _dense(kv_lens, "kv_lens", i32, (batch,), device)
    _dense(cu_q, "cu_q", i32, (batch + 1,), device)
    if out is None:
        out = torch.empty(q_shape, dtype=bf16, device=q.device)
    os = _rows(out, "out", bf16, q_shape, device)
    lse = torch.empty((q_tokens, heads), dtype=torch.float32, device=q.device) if return_lse else None
    nbytes = _attention_bytes(batch, q_tokens, heads, kv_heads, dim, k_cache.shape[1], table_width)
    _launch("lowm_paged_attention_fp8", (
        q.data_ptr(), qs[0], qs[1], *cache, page_table.data_ptr(), table_stride, table_width, kv_lens.data_ptr(),
        cu_q.data_ptr(), out.data_ptr(), os[0], os[1], None if lse is None else lse.data_ptr(), batch, q_tokens, heads, kv_heads,
        dim, 1.0 / math.sqrt(dim) if scale is None else scale, window), nbytes, device, _current_stream(device))
    return (out, lse) if return_lse else out
