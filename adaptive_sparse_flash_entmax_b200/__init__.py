"""B200-native fused alpha-entmax attention (AdaSplash-style), forward and backward.

The computation lives in ``libentattn.so`` (hand-written CUDA for sm_100a,
C ABI in ``include/entattn.h``); ``capi`` binds it with ctypes under the same
names, and ``attention`` wraps it for PyTorch tensors.  ``kvcache`` holds the paged
4-bit key/value cache and the attention of a decoder's newest tokens against it.
"""
from . import capi
from .attention import (EntmaxAttention, entmax_attention, entmax_attn_bwd, entmax_attn_fwd,
                        read_status, workspace)
from .kvcache import KV4Cache, entmax_attn_kv4, kv4_alloc, kv4_read, kv4_workspace, kv4_write

__all__ = ["capi", "EntmaxAttention", "entmax_attention", "entmax_attn_fwd", "entmax_attn_bwd",
           "read_status", "workspace", "KV4Cache", "kv4_alloc", "kv4_write", "kv4_read",
           "kv4_workspace", "entmax_attn_kv4"]
