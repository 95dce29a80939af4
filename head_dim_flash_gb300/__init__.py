"""Exact softmax attention for large head dims (D = 64..1024, tuned for 320..1024) on GB300 (sm_103a).

Forward (O and fp32 LSE) and backward (dQ, dK, dV) with bottom-right causal
masking, GQA/MQA head broadcast and packed varlen batches, computed by
hand-written tcgen05/TMA kernels behind the C ABI of ``include/ffpa.h``.
"""
from .api import (RopePlan, attention, bwd, bwd_workspace_bytes, decode_fwd, decode_fwd_kv4, decode_fwd_shared,
                  decode_fwd_weights, decode_kv4_workspace, decode_shared_workspace, decode_supported,
                  decode_weights_workspace, fp8_quantize, fwd, fwd_fp8, get_status, kv4_cache, kv4_read, kv4_write,
                  kv_evict, rope, rope_plan, varlen_attention, varlen_bwd, varlen_fwd, varlen_fwd_fp8,
                  varlen_kv4_read, varlen_kv4_write, varlen_rope)

__all__ = ["attention", "varlen_attention", "fwd", "bwd", "bwd_workspace_bytes", "varlen_fwd", "varlen_bwd",
           "decode_fwd", "decode_supported", "fwd_fp8", "varlen_fwd_fp8", "fp8_quantize", "kv4_cache", "kv4_write",
           "varlen_kv4_write", "kv4_read", "varlen_kv4_read", "decode_fwd_kv4", "decode_kv4_workspace", "RopePlan",
           "rope_plan", "rope", "varlen_rope", "decode_fwd_shared", "decode_shared_workspace", "decode_fwd_weights",
           "decode_weights_workspace", "kv_evict", "get_status"]
