"""ctypes binding of the decoder-layer operators in ``include/lowm_layer.h``.

The functions named ``lowm_*`` forward to the function of the same name in
``liblowm_gemm.so``; :func:`residual_norm`, :func:`rope_append`,
:func:`paged_attention` and :func:`moe` take torch tensors, check them, make the
outputs that are not given and launch.  There is no fallback.  Inference only:
none of them records a gradient.

``stream`` is as in :mod:`.lowm`.  A call with a stream runs as under
``with torch.cuda.stream(stream)``: the outputs and workspaces that it makes
belong to that stream, and nothing is ordered against torch's current one.
The tensors' device need not be torch's current one.
Calls on a device's default stream share one workspace that is kept between
them (:func:`release_workspaces`); they may come from several host threads.
"""
from __future__ import annotations

import ctypes
import functools
import math
import threading

import torch

from . import lowm
from .lowm import LOWM_OK, LowmError

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


# Workspace sizes follow from the sizes alone.
_attention_bytes = functools.lru_cache(maxsize=4096)(lowm_paged_attention_workspace)
_moe_bytes = functools.lru_cache(maxsize=4096)(lowm_moe_workspace)


# A call's checks are plain comparisons; what is wrong is worked out only when one fails.
def _refuse(x, name: str, dtype, shape, device: int, contiguous: bool = False):
    if x.dtype is not dtype:
        raise TypeError("%s must be %s, not %s" % (name, dtype, x.dtype))
    if x.shape != shape:
        raise ValueError("%s must be %s, not %s" % (name, tuple(shape), tuple(x.shape)))
    if not x.is_cuda or x.get_device() != device:
        raise ValueError("%s must be on cuda:%d, not %s" % (name, device, x.device))
    raise ValueError("%s must be contiguous" % name if contiguous else "the last dimension of %s must be contiguous" % name)


def _rows(x, name: str, dtype, shape, device: int):
    """Check a tensor whose last dimension must be contiguous; returns its strides."""
    strides = x.stride()
    if x.dtype is not dtype or x.shape != shape or x.get_device() != device or (strides[-1] != 1 and shape[-1] > 1):
        _refuse(x, name, dtype, shape, device)
    return strides


def _row_stride(x, name: str, dtype, shape, device: int) -> int:
    """Check a matrix; returns its row stride (of a single row, whose stride may be anything: its width)."""
    stride = _rows(x, name, dtype, shape, device)[0]
    return stride if shape[0] > 1 else shape[1]


def _dense(x, name: str, dtype, shape, device: int):
    """Check a contiguous tensor."""
    if x.dtype is not dtype or x.shape != shape or x.get_device() != device or not x.is_contiguous():
        _refuse(x, name, dtype, shape, device, True)


def _cuda(x, name: str) -> int:
    if not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    return x.get_device()


# The raw handle of torch's current stream: torch.cuda.current_stream() makes a stream object first, which
# takes longer than all checks of a call (2.9 us of a norm's 15.5 us on the host).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


# The workspace of the calls on each device's default stream.  An operator with a workspace is two launches, and ctypes
# lets other threads run during a call: the lock is held until both are enqueued, so that the stream runs all of one
# call's kernels before the next call's.  (A lock that the thread may take again: a finaliser can call an operator.)  A
# call on another stream allocates its own.  The default stream is never destroyed nor captured.  Allocated at every
# call, a workspace cost paged_attention 4 of 20 us on the host.
_kept: dict = {}
_kept_lock = threading.RLock()


def _launch(name: str, args, nbytes: int, device: int, stream: int) -> None:
    """Call the library's function `name` with `args`, `nbytes` of scratch memory and `stream`."""
    fn = function(name)
    if stream:
        own = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
        s = fn(*args, own.data_ptr(), nbytes, stream)
    else:
        with _kept_lock:
            kept = _kept.get(device)
            if kept is None or kept[1].numel() < nbytes:
                own = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", device))
                kept = _kept[device] = (own.data_ptr(), own)
            s = fn(*args, kept[0], nbytes, stream)
    if s != LOWM_OK:
        raise LowmError(s, name)


def release_workspaces() -> None:
    """Give the workspaces kept for the default streams back to torch's allocator."""
    with _kept_lock:
        _kept.clear()


def _on(stream, device: int):
    """The context in which a call on tensors of `device` runs: that device current, and `stream` if there is one.

    The library launches on the current device and takes its SM count and status word from there, whatever device the
    pointers belong to; a handle of 0 is the default stream of whichever device is current.
    """
    if stream is None:
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)
    elif stream.device.index != device:
        raise ValueError("stream must be on cuda:%d like the tensors, not %s" % (device, stream.device))
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
    ``residual`` itself.  out_residual may be ``residual``, out may be ``block``.
    """
    device = _cuda(residual, "residual")
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return residual_norm(residual, block, post_weight=post_weight, gate=gate, pre_weight=pre_weight,
                                 scale=scale, eps=eps, out_residual=out_residual, out=out)
    shape = residual.shape
    if len(shape) != 2:
        raise ValueError("residual must be [tokens, hidden]")
    bf16, dtype = torch.bfloat16, residual.dtype
    if dtype is not bf16 and dtype is not torch.float32:
        raise TypeError("residual must be bfloat16 or float32, not %s" % dtype)
    residual_stride = _rows(residual, "residual", dtype, shape, device)[0]
    tokens, hidden = shape
    gate_stride = block_stride = out_residual_stride = 0
    block_ptr = gate_ptr = post_ptr = pre_ptr = out_residual_ptr = None
    if block is not None:
        block_stride = _rows(block, "block", bf16, shape, device)[0]
        block_ptr = block.data_ptr()
        if out_residual is None:
            out_residual = torch.empty(shape, dtype=dtype, device=residual.device)
        out_residual_stride = _row_stride(out_residual, "out_residual", dtype, shape, device)
        out_residual_ptr = out_residual.data_ptr()
    elif post_weight is not None or gate is not None or out_residual is not None or scale != 1.0:
        raise ValueError("post_weight, gate, scale and out_residual need a block")
    if gate is not None:
        if gate.dim() == 1:
            _rows(gate, "gate", bf16, shape[1:], device)
        else:
            gate_stride = _rows(gate, "gate", bf16, shape, device)[0]
        gate_ptr = gate.data_ptr()
    if post_weight is not None:
        _rows(post_weight, "post_weight", bf16, shape[1:], device)
        post_ptr = post_weight.data_ptr()
    if pre_weight is not None:
        _rows(pre_weight, "pre_weight", bf16, shape[1:], device)
        pre_ptr = pre_weight.data_ptr()
    if out is None:
        out = torch.empty(shape, dtype=bf16, device=residual.device)
    out_stride = _row_stride(out, "out", bf16, shape, device)
    s = function("lowm_residual_norm")(
        residual.data_ptr(), dtype is not bf16, residual_stride, block_ptr, block_stride, post_ptr, gate_ptr,
        gate_stride, pre_ptr, out_residual_ptr, out_residual_stride, out.data_ptr(), out_stride, tokens, hidden, scale,
        eps, _current_stream(device))
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
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return rope_append(q, k, v, cos_sin, positions, slots, k_cache, v_cache, sections=sections,
                               interleaved=interleaved, out=out)
    bf16, i64 = torch.bfloat16, torch.int64
    if q.dim() != 3 or k.dim() != 3 or k_cache.dim() != 4 or v_cache.dim() != 4 or cos_sin.dim() != 2:
        raise ValueError("q and k must be [tokens, heads, dim], the caches [num_pages, page_size, kv_heads, dim] "
                         "and cos_sin [table_rows, rotary]")
    q_shape = q.shape
    tokens, heads, dim = q_shape
    kv_heads = k.shape[1]
    table_shape = cos_sin.shape
    table_rows, rotary = table_shape
    num_pages, page_size = k_cache.shape[:2]
    kv_shape, cache_shape = (tokens, kv_heads, dim), (num_pages, page_size, kv_heads, dim)
    qs = _rows(q, "q", bf16, q_shape, device)
    ks = _rows(k, "k", bf16, kv_shape, device)
    vs = _rows(v, "v", bf16, kv_shape, device)
    _dense(cos_sin, "cos_sin", torch.float32, table_shape, device)
    _dense(slots, "slots", i64, (tokens,), device)
    kc = _rows(k_cache, "k_cache", bf16, cache_shape, device)
    vc = _rows(v_cache, "v_cache", bf16, cache_shape, device)
    if positions.dim() == 1:
        axes, positions_stride = 1, 0
        _dense(positions, "positions", i64, (tokens,), device)
        if sections is not None and tuple(sections) != (rotary // 2,):
            raise ValueError("sections of one axis must be (rotary / 2,)")
        section0, section1 = rotary // 2, 0
    else:
        axes = positions.shape[0]
        positions_stride = _rows(positions, "positions", i64, (axes, tokens), device)[0]
        if sections is None or not 1 <= axes <= 3 or len(sections) != axes or sum(sections) * 2 != rotary:
            raise ValueError("positions [axes, tokens] need one to three axes and a section (rotary pairs) of each, "
                             "rotary / 2 in all")
        section0, section1 = sections[0], sections[1] if axes > 1 else 0
    if out is None:
        out = torch.empty(q_shape, dtype=bf16, device=q.device)
    os = _rows(out, "out", bf16, q_shape, device)
    s = function("lowm_rope_append")(
        q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], cos_sin.data_ptr(),
        table_rows, positions.data_ptr(), positions_stride, axes, section0, section1, interleaved, slots.data_ptr(),
        out.data_ptr(), os[0], os[1], k_cache.data_ptr(), kc[0], kc[1], kc[2], v_cache.data_ptr(), vc[0], vc[1], vc[2],
        num_pages, page_size, tokens, heads, kv_heads, dim, rotary, _current_stream(device))
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
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q, scale=scale, window=window,
                                   out=out, return_lse=return_lse)
    bf16, i32 = torch.bfloat16, torch.int32
    if q.dim() != 3 or k_cache.dim() != 4 or page_table.dim() != 2:
        raise ValueError("q must be [q_tokens, heads, dim], the caches [num_pages, page_size, kv_heads, dim] and "
                         "page_table [batch, table_width]")
    q_shape, cache_shape, table_shape = q.shape, k_cache.shape, page_table.shape
    q_tokens, heads, dim = q_shape
    num_pages, page_size, kv_heads, cache_dim = cache_shape
    batch, table_width = table_shape
    if cache_dim != dim:
        raise ValueError("q and the caches must have one head size, not %d and %d" % (dim, cache_dim))
    qs = _rows(q, "q", bf16, q_shape, device)
    kc = _rows(k_cache, "k_cache", bf16, cache_shape, device)
    vc = _rows(v_cache, "v_cache", bf16, cache_shape, device)
    table_stride = _rows(page_table, "page_table", i32, table_shape, device)[0]
    _dense(kv_lens, "kv_lens", i32, (batch,), device)
    _dense(cu_q, "cu_q", i32, (batch + 1,), device)
    if out is None:
        out = torch.empty(q_shape, dtype=bf16, device=q.device)
    os = _rows(out, "out", bf16, q_shape, device)
    lse = torch.empty((q_tokens, heads), dtype=torch.float32, device=q.device) if return_lse else None
    nbytes = _attention_bytes(batch, q_tokens, heads, kv_heads, dim)
    _launch("lowm_paged_attention", (
        q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), kc[0], kc[1], kc[2], v_cache.data_ptr(), vc[0], vc[1], vc[2],
        num_pages, page_size, page_table.data_ptr(), table_stride, table_width, kv_lens.data_ptr(), cu_q.data_ptr(),
        out.data_ptr(), os[0], os[1], None if lse is None else lse.data_ptr(), batch, q_tokens, heads, kv_heads, dim,
        1.0 / math.sqrt(dim) if scale is None else scale, window), nbytes, device, _current_stream(device))
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
    if stream is not None or _current_device() != device:
        with _on(stream, device):
            return moe(x, router_weight, gate_up, down, top_k, scoring=scoring, bias=bias, renormalize=renormalize,
                       scale=scale, out=out)
    bf16 = torch.bfloat16
    if x.dim() != 2 or router_weight.dim() != 2 or down.dim() != 3:
        raise ValueError("x must be [tokens, hidden], router_weight [experts, hidden] and down [experts, hidden, inner]")
    kind = _SCORING.get(scoring)
    if kind is None:
        raise ValueError("scoring must be 'softmax' or 'sigmoid'")
    x_shape = x.shape
    tokens, hidden = x_shape
    experts, _, inner = down.shape
    x_stride = _row_stride(x, "x", bf16, x_shape, device)
    _dense(router_weight, "router_weight", bf16, (experts, hidden), device)
    _dense(gate_up, "gate_up", bf16, (experts, 2 * inner, hidden), device)
    _dense(down, "down", bf16, (experts, hidden, inner), device)
    bias_ptr = None
    if bias is not None:
        _dense(bias, "bias", torch.float32, (experts,), device)
        bias_ptr = bias.data_ptr()
    if out is None:
        out = torch.empty(x_shape, dtype=bf16, device=x.device)
    out_stride = _row_stride(out, "out", bf16, x_shape, device)
    nbytes = _moe_bytes(tokens, hidden, inner, experts, top_k)
    _launch("lowm_moe", (
        x.data_ptr(), x_stride, router_weight.data_ptr(), bias_ptr, gate_up.data_ptr(), down.data_ptr(),
        out.data_ptr(), out_stride, tokens, hidden, inner, experts, top_k, kind, renormalize, scale),
        nbytes, device, _current_stream(device))
    return out
