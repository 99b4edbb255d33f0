"""GB300-native low-M split-K bf16 GEMM: C[M,N] = A[M,K] . W[N,K]^T, and the
decoder-layer operators around it (residual norms, rotary append, paged
attention, mixture of experts).

The compute lives in ``liblowm_gemm.so`` (CUDA C++ for sm_103a, built by
``split_bf16_gemm_swap_gb300.build``); :mod:`.lowm` (the GEMM) and
:mod:`.layer` (the layer operators, imported on first use) are its ctypes
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


def __getattr__(name):
    if name in _LAYER:
        from . import layer
        value = globals()[name] = getattr(layer, name)
        return value
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
