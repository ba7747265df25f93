"""Segment-parallel Kimi Delta Attention (KDA) forward on GB300 (sm_103a).

The compute lives in ``libkda.so`` (hand-written CUDA for sm_103a behind the C
ABI of ``include/kda.h``); ``binding`` is its thin ctypes binding, whose
functions carry the C entry points' names and are re-exported here on first
use.  Accessing any of them raises ImportError when libkda.so has not been
built: there is no fallback.  ``inputs`` draws the seeded synthetic
workloads and can be used without the library.
"""
from __future__ import annotations

import importlib

_BINDING_NAMES = ("kda_status_string", "kda_plan_segments", "kda_plan_check", "kda_plan_segments_refined", "kda_workspace_layout",
                  "kda_workspace_bytes", "kda_segment_forward", "kda_compose_summaries", "kda_apply_boundary",
                  "kda_forward_segmented", "kda_forward_two_pass", "kda_forward_segmented_noalloc",
                  "kda_device_status", "kda_selftest_wait_expiry", "kda_compose_summaries_blocked",
                  "kda_scan_workspace_bytes", "kda_backward_segmented", "kda_backward_workspace_bytes", "kda_gated_scan_forward",
                  "kda_gated_scan_backward", "kda_gated_scan_workspace_bytes", "kda_gated_scan_step", "kda_block_norm_forward",
                  "kda_block_norm_backward", "kda_block_norm_workspace_bytes", "kda_decode_step", "kda_rotary_phases",
                  "kda_head_norm_rotary_forward", "kda_head_norm_rotary_backward", "kda_head_norm_rotary_workspace_bytes",
                  "kda_window_attention_forward", "kda_window_attention_backward", "kda_window_attention_workspace_bytes", "kda_window_cache_fill", "kda_window_attention_step", "upload_plan", "KDAError", "LIB_PATH")


def __getattr__(name):
    if name in _BINDING_NAMES:
        value = globals()[name] = getattr(importlib.import_module(".binding", __name__), name)
        return value
    raise AttributeError(name)
