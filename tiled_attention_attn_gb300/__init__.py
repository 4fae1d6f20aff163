"""GB300 (sm_103a) tiled attention forward: O = softmax(scale * Q K^T [+ causal]) V
with online-softmax running statistics, and its backward (dq, dk, dv from the
kept lse), behind the C ABI of include/attn.h.

The binding loads libattn.so on first use; build it with
``tiled_attention_attn_gb300.build.build()``.
"""

from .attn import (  # noqa: F401
    AttnError,
    attn_bwd,
    attn_decode,
    attn_decode_fp8,
    attn_decode_paged,
    attn_func,
    attn_func_padded,
    attn_fwd,
    attn_fwd_paged,
    attn_tree_fp8,
    cache_append,
    cache_append_fp8,
    cache_evict,
    cache_read_fp8,
    get_error,
    key_weights,
    last_device_error,
    lib,
    plan,
    qk_norm_rotary,
    qk_norm_rotary_bwd,
    qk_norm_rotary_func,
    rotary_freqs,
    rotary_scaled,
    rotary_scaled_func,
    selftest_wait_timeout,
    set_wait_timeout_ns,
    strerror,
)
