"""Sliding-window (banded, "diagonal") attention for one NVIDIA GB300 (sm_103a).

The compute runs in hand-written CUDA kernels behind a C ABI (include/swab.h,
built into ``_lib/libswab.so`` by ``build.build()``); this package is the thin
ctypes binding over it plus the seeded input generators.  Nothing here
computes attention on the host.
"""
from ._binding import (API_FUNCTIONS, Desc, SwabError, add_bias_transpose,  # noqa: F401
                       band_attention,
                       band_attention_bwd, band_attention_bwd_noalloc,
                       band_attention_bwd_workspace, band_attention_dropout_mask_bytes, band_pv,
                       band_pv_bwd_t, band_qk, band_qk_bwd_t, band_softmax, band_softmax_bwd,
                       band_softmax_dropout,
                       device_status, global_attention, global_attention_bwd,
                       global_attention_workspace, library_path, load, selftest_wait_timeout,
                       bounds_checked, bounds_report, selftest_bounds,
                       status_string, version)
from .serve import (CacheDesc, DecodeDesc, RotaryDesc, band_decode,  # noqa: F401
                    band_decode_workspace, cache_slots, rotary, rotary_append, rotary_bwd,
                    rotary_frequencies)
from .norm import (NormDesc, norm_rotary, norm_rotary_append, norm_rotary_bwd,  # noqa: F401
                   norm_rotary_bwd_workspace)
from .cache4 import (band_decode4, band_decode4_workspace, cache4_shapes, cache_read4,  # noqa: F401
                     rotary_append4)
from .decode_loop import DecodeLoop  # noqa: F401
from .inputs import WORKLOADS, Workload, seeded_qkvo, workload_inputs  # noqa: F401

__all__ = ["Desc", "SwabError", "add_bias_transpose", "band_qk", "band_softmax",
           "band_softmax_dropout", "band_pv", "band_qk_bwd_t", "global_attention",
           "global_attention_bwd", "global_attention_workspace",
           "band_pv_bwd_t", "band_softmax_bwd", "band_attention", "band_attention_bwd",
           "band_attention_bwd_noalloc",
           "band_attention_bwd_workspace", "band_attention_dropout_mask_bytes", "device_status", "selftest_wait_timeout", "bounds_checked", "bounds_report",
           "selftest_bounds", "load",
           "CacheDesc", "DecodeDesc", "DecodeLoop", "RotaryDesc", "rotary_frequencies", "rotary", "rotary_bwd",
           "cache_slots", "rotary_append", "band_decode", "band_decode_workspace",
           "NormDesc", "norm_rotary", "norm_rotary_bwd", "norm_rotary_bwd_workspace", "norm_rotary_append",
           "rotary_append4", "cache_read4", "cache4_shapes", "band_decode4", "band_decode4_workspace",
           "library_path", "version", "status_string", "WORKLOADS", "Workload",
           "seeded_qkvo", "workload_inputs"]
