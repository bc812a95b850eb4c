"""GB300 (sm_103a) multi-head scaled dot-product attention forward.

``mha_fwd`` computes softmax(Q K^T * scale) V per (batch, head) on hand-written
CUDA kernels: a tcgen05/TMA/TMEM kernel for long sequences, a packed
tensor-core kernel for sentence-length sequences, and an fp32 CUDA-core
kernel.  Masks: causal, key padding, query padding (see include/mha.h).
``mha_fwd_ex`` adds shared key/value heads (grouped- and multi-query
attention) and the [B, L, H, d] layout; ``mha_sublayer_fwd`` runs the whole
multi-head sublayer (projections with biases on ``mha_linear_fwd``'s tensor-core
kernel, attention, output projection).

For generation from a paged key/value cache and for the layers around it:
``mha_qk_norm_rope_fwd`` / ``_bwd`` (per-head norm and position rotation),
``mha_paged_append`` and ``mha_paged_fwd``; ``mha_paged_append_at`` and
``mha_paged_tree_fwd`` for trees of drafted tokens; ``mha_paged_reserve``,
``mha_paged_copy`` and ``mha_paged_compact`` for the pages under them (see
include/mha_paged.h).
"""
from .mha import (MHA_DTYPE_BF16, MHA_DTYPE_F32, MHA_ERR_CUDA, MHA_ERR_INVALID_ARGUMENT,
                  MHA_ERR_TIMEOUT, MHA_ERR_UNSUPPORTED, MHA_MASK_CAUSAL, MHA_MASK_KEY_PADDING,
                  MHA_LAYOUT_BHSD, MHA_LAYOUT_BSHD, MHA_MASK_CAUSAL_TAIL, MHA_MASK_NONE,
                  MHA_MASK_QUERY_PADDING, MHA_OK, PATH_NAMES, LIB_PATH, MhaError,
                  lib, mha_debug_set_wait, mha_debug_status, mha_fwd, mha_fwd_lse, mha_fwd_ex, mha_fwd_path, mha_fwd_path_ex,
                  mha_linear_fwd,
                  mha_sublayer_fwd, mha_sublayer_fwd_static, mha_sublayer_workspace_size,
                  mha_bwd, mha_bwd_workspace_size, mha_status_string, mha_version)
from .paged import (MHA_ROPE_HALVES, MHA_ROPE_INTERLEAVED, PAGED_PATH_NAMES, mha_paged_append,
                    mha_paged_append_at, mha_paged_compact, mha_paged_copy, mha_paged_fwd,
                    mha_paged_path, mha_paged_reserve, mha_paged_reserve_workspace_size,
                    mha_paged_tree_fwd, mha_paged_workspace_size, mha_qk_norm_rope_bwd,
                    mha_qk_norm_rope_bwd_workspace_size, mha_qk_norm_rope_fwd, rope_inv_freq,
                    tree_mask)

__all__ = ["mha_fwd", "mha_fwd_ex", "mha_fwd_lse", "mha_linear_fwd", "mha_sublayer_fwd", "mha_bwd",
           "mha_bwd_workspace_size",
           "mha_sublayer_fwd_static",
           "mha_sublayer_workspace_size", "mha_fwd_path", "mha_fwd_path_ex", "mha_status_string", "mha_debug_status",
           "mha_debug_set_wait", "mha_version",
           "MhaError", "lib", "LIB_PATH", "PATH_NAMES", "MHA_OK", "MHA_ERR_INVALID_ARGUMENT",
           "MHA_ERR_UNSUPPORTED", "MHA_ERR_CUDA", "MHA_ERR_TIMEOUT", "MHA_DTYPE_F32",
           "MHA_DTYPE_BF16", "MHA_MASK_NONE", "MHA_MASK_CAUSAL", "MHA_MASK_KEY_PADDING",
           "MHA_MASK_QUERY_PADDING", "MHA_MASK_CAUSAL_TAIL", "MHA_LAYOUT_BHSD",
           "MHA_LAYOUT_BSHD", "MHA_ROPE_HALVES", "MHA_ROPE_INTERLEAVED", "PAGED_PATH_NAMES",
           "mha_qk_norm_rope_fwd", "mha_qk_norm_rope_bwd", "mha_qk_norm_rope_bwd_workspace_size",
           "mha_paged_append", "mha_paged_append_at", "mha_paged_fwd", "mha_paged_tree_fwd",
           "mha_paged_path", "mha_paged_workspace_size", "rope_inv_freq", "tree_mask",
           "mha_paged_reserve", "mha_paged_reserve_workspace_size", "mha_paged_copy",
           "mha_paged_compact"]
