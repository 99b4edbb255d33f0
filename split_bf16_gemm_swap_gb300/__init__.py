"""GB300-native low-M split-K bf16 GEMM: C[M,N] = A[M,K] . W[N,K]^T, and the
decoder-layer operators around it (residual norms, rotary append, paged
attention, mixture of experts), the 8-bit forms of the GEMM and of the paged
cache, and the bookkeeping of the cache's pages.

The compute lives in ``liblowm_gemm.so`` (CUDA C++ for sm_103a, built by
``split_bf16_gemm_swap_gb300.build``); :mod:`.lowm` (the GEMM),
:mod:`.layer` (the layer operators), :mod:`.fp8` (the 8-bit forms) and
:mod:`.pages` (pages; these three imported on first use) are its ctypes
bindings and :mod:`.inputs` draws the seeded synthetic operands.  Importing the
package does not load the library; the first call does, and fails loudly if it
is missing.
"""
from .lowm import (  # noqa: F401
    ABI_FUNCTIONS, LOWM_FLAG_A_BEFORE_PDL_WAIT, LOWM_FLAG_W_BEFORE_PDL_WAIT, LOWM_OK, LowmError, gemm,
    lowm_gemm_bf16, lowm_gemm_bf16_debug, lowm_gemm_bf16_ex, lowm_gemm_bf16_host,
    lowm_gemm_query_tactic, lowm_gemm_query_tactic_ex, lowm_gemm_sync_status, lowm_status_string, lowm_tmem_hog_launch,
)

_LAYER = ("LOWM_MOE_SIGMOID", "LOWM_MOE_SOFTMAX", "moe", "paged_attention", "release_workspaces", "residual_norm",
          "rope_append", "lowm_moe", "lowm_moe_workspace", "lowm_paged_attention", "lowm_paged_attention_workspace",
          "lowm_residual_norm", "lowm_rope_append")


_FP8 = ("gemm_fp8", "paged_attention_fp8", "quantize_fp8", "rope_append_fp8", "lowm_gemm_fp8",
        "lowm_gemm_fp8_bf16", "lowm_gemm_fp8_bf16_workspace", "lowm_paged_attention_fp8",
        "lowm_paged_attention_fp8_workspace", "lowm_quantize_fp8", "lowm_rope_append_fp8")
_PAGES = ("compact_pages", "copy_pages", "extend_pages", "fork_pages", "lowm_compact_pages", "lowm_compact_pages_workspace",
          "lowm_copy_pages", "lowm_extend_pages", "lowm_extend_pages_workspace", "lowm_fork_pages", "lowm_page_span_t")
_MODULES = {name: module for module, names in (("layer", _LAYER), ("fp8", _FP8), ("pages", _PAGES)) for name in names}


def __getattr__(name):
    if name in _MODULES:
        import importlib
        value = globals()[name] = getattr(importlib.import_module("." + _MODULES[name], __name__), name)
        return value
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
