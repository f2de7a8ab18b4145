"""GB300-native (sm_103a) exact IO-aware attention.

The compute lives in libattn_gb300.so (C ABI in include/attn.h): tcgen05 tensor-core kernels
for fp16/bf16 and CUDA-core kernels for fp32.  This package is the thin PyTorch binding.
"""
from .attention import (bwd, bwd_cross, bwd_varlen, bwd_varlen_gqa, flash_attention, flash_attn_varlen_gqa_func,
                        flash_attn_varlen_qkvpacked_func, fwd, fwd_kvcache, fwd_kvcache8, fwd_kvpages, fwd_varlen,
                        fwd_varlen_gqa, get_device_status, kvcache8_append, kvcache8_workspace_bytes, kvcache_evict,
                        kvcache_weights, kvcache_workspace_bytes, kvpages_append, kvpages_compact, kvpages_copy,
                        kvpages_fork, kvpages_free, kvpages_reserve, kvpages_workspace_bytes)
from ._lib import AttnError

__all__ = ["flash_attention", "flash_attn_varlen_qkvpacked_func", "fwd", "bwd", "fwd_varlen", "bwd_varlen",
           "fwd_kvcache", "kvcache_workspace_bytes", "kvcache8_append", "fwd_kvcache8", "kvcache8_workspace_bytes",
           "kvcache_weights", "kvcache_evict", "fwd_varlen_gqa", "bwd_varlen_gqa", "flash_attn_varlen_gqa_func",
           "kvpages_append", "fwd_kvpages", "kvpages_workspace_bytes", "kvpages_free", "kvpages_fork", "kvpages_reserve",
           "kvpages_compact", "kvpages_copy", "bwd_cross", "get_device_status", "AttnError"]
