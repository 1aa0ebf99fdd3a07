"""exact_attention_69_gb300: the fused exact-attention forward pass,
softmax(scale * Q K^T [+ mask]) V, as hand-written sm_103a (GB300) kernels
behind a small C ABI (include/attn.h, libattn.so).

Masks: none, causal (tiles above the diagonal skipped), neighbourhood attention
on 2-D grids and 3-D volumes with clamped or circular ("wrap") windows chosen
per axis, and dilation (tiles no window touches skipped). Outputs: O in bf16
and the fp32 log-sum-exp. attn_bwd / attention: the backward pass for every
mask. tune: the split-KV schedule chosen by measurement.

For language models: qk_norm_rope (per-head norm and rotary positions, with
gradients), kv_append (new keys and values into a paged cache, normed and
rotated on the way) and attn_paged (attention over such a cache, with a prefix
that the batch shares). For long caches: kv_bounds, block_scores, block_select
and attn_blocks (attention over the pages that a cheap score selects for each
query), kv_weights and kv_evict (a cache cut to the tokens that received the most
attention).
"""
from .api import (  # noqa: F401
    attention, attn_bwd, attn_fwd, device_status, na2d, na3d, sm_count, tune, workspace_bytes)
from .cache import (  # noqa: F401
    attn_paged, kv_append, qk_norm_rope, qk_norm_rope_bwd, qk_norm_rope_fwd, rope_freqs)
from .long_cache import (  # noqa: F401
    attn_blocks, block_scores, block_select, kv_bounds, kv_evict, kv_weights)
from ._lib import AttnError  # noqa: F401

__all__ = ["attn_fwd", "attn_bwd", "attention", "na2d", "na3d", "tune", "device_status", "sm_count",
           "workspace_bytes", "qk_norm_rope", "qk_norm_rope_fwd", "qk_norm_rope_bwd", "rope_freqs",
           "kv_append", "attn_paged", "kv_bounds", "block_scores", "block_select", "attn_blocks", "kv_weights",
           "kv_evict", "AttnError"]
