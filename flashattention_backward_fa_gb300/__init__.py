"""GB300-native (sm_103a) FlashAttention forward and backward.

The computation lives in libfa.so, a C-ABI CUDA library (include/fa.h); this
package is its thin Python binding plus the seeded input generator used by the
tests and the bench. The library is loaded on first use and its absence is an
error: there is no CPU path.
"""
from .binding import (FA_BF16, FA_BWD_DKDV, FA_BWD_DQ, FA_BWD_PREPROCESS, FA_DQ_ATOMIC, FA_DQ_DETERMINISTIC,
                      FA_DQ_ORDERED, FA_DQ_RECOMPUTE, FA_F16, FA_F32, FaError, FaStrides,
                      alloc_workspace, attention_backward, attention_forward, default_scale, fa_bwd, fa_bwd_host,
                      fa_bwd_host_buffer_size,
                      fa_bwd_noalloc, fa_bwd_stage, fa_bwd_workspace_size, fa_fwd, fa_get_device_status,
                      fa_kv8_attn, fa_kv8_attn_workspace_size, fa_kv8_norm_rope_append, fa_qk_norm_rope_bwd,
                      fa_qk_norm_rope_bwd_workspace_size, fa_qk_norm_rope_fwd, fa_selftest_timeout,
                      fa_strerror, fa_varlen_bwd, fa_varlen_bwd_workspace_size, fa_varlen_fwd, flash_attn_func,
                      flash_attn_varlen_func, header_functions, Kv8Cache, kv8_append, kv8_attention,
                      kv8_cache_alloc, kv8_norm_rope_append, load_library, qk_norm_rope_backward,
                      qk_norm_rope_forward, qk_norm_rope_func, rope_tables, varlen_attention_backward, varlen_attention_forward)

__all__ = ["FA_BF16", "FA_BWD_DKDV", "FA_BWD_DQ", "FA_BWD_PREPROCESS", "FA_DQ_ATOMIC", "FA_DQ_DETERMINISTIC",
           "FA_DQ_ORDERED", "FA_DQ_RECOMPUTE", "FA_F16", "FA_F32", "FaError", "FaStrides",
           "alloc_workspace", "attention_backward", "attention_forward", "default_scale", "fa_bwd", "fa_bwd_host",
           "fa_bwd_host_buffer_size", "fa_bwd_noalloc", "fa_bwd_stage",
           "fa_bwd_workspace_size", "fa_fwd", "fa_get_device_status", "fa_selftest_timeout", "fa_strerror",
           "fa_varlen_bwd",
           "fa_varlen_bwd_workspace_size", "fa_varlen_fwd", "flash_attn_func", "flash_attn_varlen_func", "header_functions", "load_library",
           "fa_kv8_attn", "fa_kv8_attn_workspace_size", "fa_kv8_norm_rope_append", "fa_qk_norm_rope_bwd",
           "fa_qk_norm_rope_bwd_workspace_size", "fa_qk_norm_rope_fwd", "Kv8Cache", "kv8_append", "kv8_attention",
           "kv8_cache_alloc", "kv8_norm_rope_append", "qk_norm_rope_backward", "qk_norm_rope_forward",
           "qk_norm_rope_func", "rope_tables",
           "varlen_attention_backward", "varlen_attention_forward"]
