"""GB300 (sm_103a) Kimi Delta Attention chunked prefill forward.

Public API (thin ctypes binding of ``include/kda.h``):
  kda_fwd, kda_workspace_size, kda_read_device_status, fwd, kda_fwd_no_alloc,
  kda_fwd_host (host buffers), kda_fwd_host_device_bytes, kda_decode (one token per sequence),
  kda_fwd_schedule (the launch schedule for a unit count), kda_fwd_set_trace (chain trace),
and the token mixers beside KDA in a hybrid stack: kda_qk_norm_rope (norm and rotation of q and k),
  kda_attn_fwd (causal attention: prompts and caches), kda_lin_fwd / kda_lin_decode (linear attention
  with a decay for each head: prompts and one token per sequence), kda_attn_workspace_size,
  kda_lin_workspace_size
"""
from .binding import (KDA_FLAG_ROPE_INTERLEAVED, KDAError, fwd, kda_attn_fwd, kda_attn_workspace_size, kda_decode,  # noqa: F401
                      kda_fwd, kda_fwd_host, kda_fwd_host_device_bytes,
                      kda_fwd_host_workspace_offset, kda_fwd_no_alloc, kda_fwd_schedule, kda_fwd_set_trace,
                      kda_lin_decode, kda_lin_fwd, kda_lin_workspace_size, kda_qk_norm_rope, kda_read_device_status,
                      kda_workspace_size, load, library_path)

__all__ = ["KDA_FLAG_ROPE_INTERLEAVED", "KDAError", "fwd", "kda_attn_fwd", "kda_attn_workspace_size", "kda_decode", "kda_fwd", "kda_fwd_host", "kda_fwd_host_device_bytes", "kda_fwd_host_workspace_offset",
           "kda_fwd_no_alloc", "kda_fwd_schedule", "kda_fwd_set_trace", "kda_lin_decode", "kda_lin_fwd",
           "kda_lin_workspace_size", "kda_qk_norm_rope", "kda_read_device_status", "kda_workspace_size", "load", "library_path"]
