"""ctypes binding of the decoder-layer operators in ``include/lowm_layer.h``.

The functions named ``lowm_*`` forward to the function of the same name in
``liblowm_gemm.so``; :func:`residual_norm`, :func:`rope_append`,
:func:`paged_attention` and :func:`moe` take torch tensors, check them, make the
outputs that are not given and launch.  There is no fallback.  Inference only:
none of them records a gradient.

``stream`` is as in :mod:`.lowm`.  A call with a stream runs as under
``with torch.cuda.stream(stream)``: the outputs and workspaces that it makes
belong to that stream, and nothing is ordered against torch's current one.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import lowm
from .lowm import LOWM_OK, LowmError, _ptr, _stream

LOWM_MOE_SOFTMAX = 0
LOWM_MOE_SIGMOID = 1

# Exported C functions, in header order.
ABI_FUNCTIONS = (
    "lowm_residual_norm",
    "lowm_rope_append",
    "lowm_paged_attention",
    "lowm_paged_attention_workspace",
    "lowm_moe",
    "lowm_moe_workspace",
)

_p, _i, _l, _f, _z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_ARGTYPES = {
    "lowm_residual_norm": [_p, _i, _l, _p, _l, _p, _p, _l, _p, _p, _l, _p, _l, _i, _i, _f, _f, _p],
    "lowm_rope_append": [_p, _l, _l, _p, _l, _l, _p, _l, _l, _p, _l, _p, _l, _i, _i, _i, _i, _p, _p, _l, _l,
                         _p, _l, _l, _l, _p, _l, _l, _l, _l, _i, _i, _i, _i, _i, _i, _p],
    "lowm_paged_attention": [_p, _l, _l, _p, _l, _l, _l, _p, _l, _l, _l, _l, _i, _p, _l, _i, _p, _p, _p, _l, _l, _p,
                             _i, _i, _i, _i, _i, _f, _i, _p, _z, _p],
    "lowm_paged_attention_workspace": [_i, _i, _i, _i, _i],
    "lowm_moe": [_p, _l, _p, _p, _p, _p, _p, _l, _i, _i, _i, _i, _i, _i, _i, _f, _p, _z, _p],
    "lowm_moe_workspace": [_i, _i, _i, _i, _i],
}

_functions = {}


def function(name: str):
    """The library's function `name` with its argument types set; raises if the library is missing."""
    fn = _functions.get(name)
    if fn is None:
        fn = getattr(lowm.lib(), name)
        fn.argtypes = _ARGTYPES[name]
        fn.restype = _z if name.endswith("_workspace") else _i
        _functions[name] = fn
    return fn


def lowm_residual_norm(*args) -> int:
    return function("lowm_residual_norm")(*args)


def lowm_rope_append(*args) -> int:
    return function("lowm_rope_append")(*args)


def lowm_paged_attention(*args) -> int:
    return function("lowm_paged_attention")(*args)


def lowm_paged_attention_workspace(batch: int, q_tokens: int, heads: int, kv_heads: int, dim: int) -> int:
    return function("lowm_paged_attention_workspace")(batch, q_tokens, heads, kv_heads, dim)


def lowm_moe(*args) -> int:
    return function("lowm_moe")(*args)


def lowm_moe_workspace(tokens: int, hidden: int, inner: int, experts: int, top_k: int) -> int:
    return function("lowm_moe_workspace")(tokens, hidden, inner, experts, top_k)


def _check(x, name: str, dtype, shape, device, contiguous: bool = False):
    """One tensor argument: its type, shape, place and (at least) its innermost stride."""
    if x.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, x.dtype))
    if x.shape != shape:
        raise ValueError("%s must be %s, not %s" % (name, tuple(shape), tuple(x.shape)))
    if x.device != device:
        raise ValueError("%s must be on %s, not %s" % (name, device, x.device))
    if contiguous:
        if not x.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    elif shape and x.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)


def _cuda(x, name: str):
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return x.device


def _on(stream, device):
    """The context in which a call with an explicit stream runs."""
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def residual_norm(residual, block=None, *, post_weight=None, gate=None, pre_weight=None, scale: float = 1.0,
                  eps: float = 1e-6, out_residual=None, out=None, stream=None):
    """The norms after and before a block with its gate and the residual scale.

    ``new = scale * residual + gate * RMS(block; post_weight)``,
    ``normed = RMS(new; pre_weight)``; returns ``(new, normed)``.

    residual [tokens, hidden] bf16 or fp32 (the type of ``new``); block
    [tokens, hidden] bf16; gate [hidden] or [tokens, hidden] bf16; weights
    [hidden] bf16.  post_weight None: the block's output is not normed;
    pre_weight None: 1.  Without a block only the norm is taken and ``new`` is
    ``residual`` itself.  out_residual may be ``residual``.
    """
    device = _cuda(residual, "residual")
    if stream is not None:
        with _on(stream, device):
            return residual_norm(residual, block, post_weight=post_weight, gate=gate, pre_weight=pre_weight,
                                 scale=scale, eps=eps, out_residual=out_residual, out=out)
    shape = residual.shape
    if len(shape) != 2:
        raise ValueError("residual must be [tokens, hidden]")
    f32 = residual.dtype is torch.float32
    if not f32 and residual.dtype is not torch.bfloat16:
        raise TypeError("residual must be bfloat16 or float32, not %s" % residual.dtype)
    _check(residual, "residual", residual.dtype, shape, device)
    tokens, hidden = shape
    bf16 = torch.bfloat16
    gate_stride = block_stride = out_residual_stride = 0
    if block is not None:
        _check(block, "block", bf16, shape, device)
        block_stride = block.stride(0)
        if out_residual is None:
            out_residual = torch.empty(shape, dtype=residual.dtype, device=device)
        else:
            _check(out_residual, "out_residual", residual.dtype, shape, device)
        out_residual_stride = out_residual.stride(0) if tokens > 1 else hidden
    elif post_weight is not None or gate is not None or out_residual is not None or scale != 1.0:
        raise ValueError("post_weight, gate, scale and out_residual need a block")
    if gate is not None:
        if gate.dim() == 1:
            _check(gate, "gate", bf16, shape[1:], device)
        else:
            _check(gate, "gate", bf16, shape, device)
            gate_stride = gate.stride(0)
    if post_weight is not None:
        _check(post_weight, "post_weight", bf16, shape[1:], device)
    if pre_weight is not None:
        _check(pre_weight, "pre_weight", bf16, shape[1:], device)
    if out is None:
        out = torch.empty(shape, dtype=bf16, device=device)
    else:
        _check(out, "out", bf16, shape, device)
    s = function("lowm_residual_norm")(
        residual.data_ptr(), f32, residual.stride(0), _ptr(block), block_stride, _ptr(post_weight), _ptr(gate),
        gate_stride, _ptr(pre_weight), _ptr(out_residual), out_residual_stride, out.data_ptr(),
        out.stride(0) if tokens > 1 else hidden, tokens, hidden, scale, eps, _stream(None))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_residual_norm")
    return (residual if block is None else out_residual), out


def rope_append(q, k, v, cos_sin, positions, slots, k_cache, v_cache, *, sections=None, interleaved: bool = False,
                out=None, stream=None):
    """Rotary positions for q and k, and the append of k and v to the paged cache; returns the rotated q.

    q [tokens, heads, dim], k and v [tokens, kv_heads, dim] bf16 (slices of one
    projection will do); cos_sin [table_rows, rotary] fp32, cosines then sines;
    positions int64 [tokens], or [axes, tokens] with `sections` (rotary pairs
    per axis); slots int64 [tokens], page * page_size + place, negative for
    padding; k_cache, v_cache [num_pages, page_size, kv_heads, dim] bf16.
    `out` may be q.
    """
    device = _cuda(q, "q")
    if stream is not None:
        with _on(stream, device):
            return rope_append(q, k, v, cos_sin, positions, slots, k_cache, v_cache, sections=sections,
                               interleaved=interleaved, out=out)
    bf16 = torch.bfloat16
    if q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4 or v_cache.dim() != 4 or cos_sin.dim() != 2:
        raise ValueError("q and k must be [tokens, heads, dim], the caches [num_pages, page_size, kv_heads, dim] "
                         "and cos_sin [table_rows, rotary]")
    tokens, heads, dim = q.shape
    kv_heads = k.shape[1]
    table_rows, rotary = cos_sin.shape
    num_pages, page_size = k_cache.shape[:2]
    _check(q, "q", bf16, q.shape, device)
    _check(k, "k", bf16, (tokens, kv_heads, dim), device)
    _check(v, "v", bf16, k.shape, device)
    _check(cos_sin, "cos_sin", torch.float32, cos_sin.shape, device, True)
    _check(slots, "slots", torch.int64, (tokens,), device, True)
    _check(k_cache, "k_cache", bf16, (num_pages, page_size, kv_heads, dim), device)
    _check(v_cache, "v_cache", bf16, k_cache.shape, device)
    if positions.dim() == 1:
        axes, positions_stride = 1, 0
        _check(positions, "positions", torch.int64, (tokens,), device)
        if sections is not None and tuple(sections) != (rotary // 2,):
            raise ValueError("sections of one axis must be (rotary / 2,)")
        sections = (rotary // 2,)
    else:
        axes = positions.shape[0]
        _check(positions, "positions", torch.int64, (axes, tokens), device)
        positions_stride = positions.stride(0)
        if sections is None or not 1 <= axes <= 3 or len(sections) != axes or sum(sections) * 2 != rotary:
            raise ValueError("positions [axes, tokens] need one to three axes and a section (rotary pairs) of each, "
                             "rotary / 2 in all")
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=bf16, device=device)
    else:
        _check(out, "out", bf16, q.shape, device)
    kc, vc = k_cache.stride(), v_cache.stride()
    qs, ks, vs, os = q.stride(), k.stride(), v.stride(), out.stride()
    s = function("lowm_rope_append")(
        _ptr(q), qs[0], qs[1], _ptr(k), ks[0], ks[1], _ptr(v), vs[0], vs[1], _ptr(cos_sin), table_rows,
        _ptr(positions), positions_stride, axes, sections[0], sections[1] if axes > 1 else 0, interleaved, _ptr(slots),
        _ptr(out), os[0], os[1], _ptr(k_cache), kc[0], kc[1], kc[2], _ptr(v_cache), vc[0], vc[1], vc[2], num_pages,
        page_size, tokens, heads, kv_heads, dim, rotary, _stream(None))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_rope_append")
    return out


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q, *, scale=None, window: int = 0, out=None,
                    return_lse: bool = False, stream=None):
    """Attention of each sequence's newest tokens over its paged keys and values.

    q [q_tokens, heads, dim] bf16, the new tokens of all sequences one after
    another (cu_q int32 [batch + 1] their starts); kv_lens int32 [batch] counts
    a sequence's tokens in the cache, the new ones included; page_table int32
    [batch, table_width].  New token i of a sequence sees the keys up to its
    own, the last `window` of them when window > 0.  scale defaults to
    dim ** -0.5.  Returns out, or (out, lse fp32 [q_tokens, heads]).
    """
    device = _cuda(q, "q")
    if stream is not None:
        with _on(stream, device):
            return paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q, scale=scale, window=window,
                                   out=out, return_lse=return_lse)
    bf16, i32 = torch.bfloat16, torch.int32
    if q.dim() != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("q must be [q_tokens, heads, dim], the caches [num_pages, page_size, kv_heads, dim] and "
                         "page_table [batch, table_width]")
    q_tokens, heads, dim = q.shape
    num_pages, page_size, kv_heads, _ = k_cache.shape
    batch, table_width = page_table.shape
    _check(q, "q", bf16, q.shape, device)
    _check(k_cache, "k_cache", bf16, (num_pages, page_size, kv_heads, dim), device)
    _check(v_cache, "v_cache", bf16, k_cache.shape, device)
    _check(page_table, "page_table", i32, page_table.shape, device)
    _check(kv_lens, "kv_lens", i32, (batch,), device, True)
    _check(cu_q, "cu_q", i32, (batch + 1,), device, True)
    if out is None:
        out = torch.empty((q_tokens, heads, dim), dtype=bf16, device=device)
    else:
        _check(out, "out", bf16, q.shape, device)
    lse = torch.empty((q_tokens, heads), dtype=torch.float32, device=device) if return_lse else None
    nbytes = lowm_paged_attention_workspace(batch, q_tokens, heads, kv_heads, dim)
    work = torch.empty(nbytes, dtype=torch.uint8, device=device)
    kc, vc, qs, os = k_cache.stride(), v_cache.stride(), q.stride(), out.stride()
    s = function("lowm_paged_attention")(
        _ptr(q), qs[0], qs[1], _ptr(k_cache), kc[0], kc[1], kc[2], _ptr(v_cache), vc[0], vc[1], vc[2], num_pages,
        page_size, _ptr(page_table), page_table.stride(0), table_width, _ptr(kv_lens), _ptr(cu_q), _ptr(out), os[0],
        os[1], _ptr(lse), batch, q_tokens, heads, kv_heads, dim, 1.0 / math.sqrt(dim) if scale is None else scale,
        window, _ptr(work), nbytes, _stream(None))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_paged_attention")
    return (out, lse) if return_lse else out


_SCORING = {"softmax": LOWM_MOE_SOFTMAX, "sigmoid": LOWM_MOE_SIGMOID}


def moe(x, router_weight, gate_up, down, top_k: int, *, scoring: str = "softmax", bias=None, renormalize: bool = True,
        scale: float = 1.0, out=None, stream=None):
    """A mixture-of-experts layer for at most 128 tokens.

    x [tokens, hidden] bf16; router_weight [experts, hidden] bf16; gate_up
    [experts, 2 * inner, hidden] bf16 (gate rows, then up rows); down [experts,
    hidden, inner] bf16; bias fp32 [experts] enters the choice of the experts
    only.  The chosen experts' scores (softmax or sigmoid of the router's
    logits), divided by their sum when `renormalize`, times `scale`, weigh the
    experts' outputs down . (silu(gate . x) * (up . x)).
    """
    device = _cuda(x, "x")
    if stream is not None:
        with _on(stream, device):
            return moe(x, router_weight, gate_up, down, top_k, scoring=scoring, bias=bias, renormalize=renormalize,
                       scale=scale, out=out)
    bf16 = torch.bfloat16
    if x.dim() != 2 or router_weight.dim() != 2 or down.dim() != 3:
        raise ValueError("x must be [tokens, hidden], router_weight [experts, hidden] and down [experts, hidden, inner]")
    if scoring not in _SCORING:
        raise ValueError("scoring must be 'softmax' or 'sigmoid'")
    tokens, hidden = x.shape
    experts, _, inner = down.shape
    _check(x, "x", bf16, x.shape, device)
    _check(router_weight, "router_weight", bf16, (experts, hidden), device, True)
    _check(gate_up, "gate_up", bf16, (experts, 2 * inner, hidden), device, True)
    _check(down, "down", bf16, (experts, hidden, inner), device, True)
    if bias is not None:
        _check(bias, "bias", torch.float32, (experts,), device, True)
    if out is None:
        out = torch.empty((tokens, hidden), dtype=bf16, device=device)
    else:
        _check(out, "out", bf16, x.shape, device)
    nbytes = lowm_moe_workspace(tokens, hidden, inner, experts, top_k)
    work = torch.empty(nbytes, dtype=torch.uint8, device=device)
    s = function("lowm_moe")(
        _ptr(x), x.stride(0) if tokens > 1 else hidden, _ptr(router_weight), _ptr(bias), _ptr(gate_up), _ptr(down), _ptr(out),
        out.stride(0) if tokens > 1 else hidden, tokens, hidden, inner, experts, top_k, _SCORING[scoring],
        renormalize, scale, _ptr(work), nbytes, _stream(None))
    if s != LOWM_OK:
        raise LowmError(s, "lowm_moe")
    return out
