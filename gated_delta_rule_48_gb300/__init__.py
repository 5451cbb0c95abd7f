"""Kimi Delta Attention (KDA) on one GB300: a C-ABI CUDA library and its Python binding.

``kda_chunk_fwd``   chunk-parallel prefill of the gated delta-rule layer.
``kda_decode_step`` single-token recurrent decode, state updated in place.

The compiled library (``csrc/`` -> ``libkda.so``) is loaded lazily on first
use; importing this package does not require a GPU.
"""
from .binding import (  # noqa: F401
    KdaError,
    build,
    kda_add_rms_norm,
    kda_add_rms_norm_quant,
    kda_attention_fwd,
    kda_chunk_fwd,
    kda_decode_step,
    kda_get_device_error,
    kda_kv4_attention,
    kda_kv4_cache,
    kda_kv4_read,
    kda_kv4_write,
    kda_matmul_fp8,
    kda_short_conv_fwd,
    kda_short_conv_step,
    kda_ssm_scan_fwd,
    kda_ssm_scan_step,
    library_path,
    load,
)

__all__ = ["KdaError", "build", "kda_add_rms_norm", "kda_add_rms_norm_quant", "kda_attention_fwd",
           "kda_chunk_fwd", "kda_decode_step", "kda_get_device_error", "kda_kv4_attention",
           "kda_kv4_cache", "kda_kv4_read", "kda_kv4_write", "kda_matmul_fp8", "kda_short_conv_fwd",
           "kda_short_conv_step", "kda_ssm_scan_fwd",
           "kda_ssm_scan_step", "library_path", "load"]
