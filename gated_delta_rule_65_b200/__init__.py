"""B200-native (sm_100a) Gated Delta Rule-2 sequence mixer.

The kernels live in ``libgdr2.so`` (sources in ``csrc/``, C ABI in ``include/gdr2.h``); ``gdr2`` is
the ctypes binding and ``workloads`` draws seeded synthetic inputs.
"""
from .gdr2 import (GDR2Error, alloc_workspace, alloc_workspace_gva, alloc_workspace_varlen,  # noqa: F401
                   attn_decode, attn_prologue_bwd, attn_prologue_cache, attn_prologue_fwd, check, chunk_bwd,
                   chunk_bwd_gva, chunk_bwd_varlen, chunk_fwd, chunk_fwd_gva, chunk_fwd_varlen, decode_step,
                   gate_prologue_bwd, gate_prologue_fwd, kv_compact, kv_fork, kv_reserve, lib, rope_freqs,
                   status_string, workspace_bytes, workspace_bytes_gva, workspace_bytes_varlen)

__all__ = ["GDR2Error", "alloc_workspace", "alloc_workspace_gva", "alloc_workspace_varlen", "attn_decode",
           "attn_prologue_bwd", "attn_prologue_cache", "attn_prologue_fwd", "check", "chunk_bwd", "chunk_bwd_gva",
           "chunk_bwd_varlen", "chunk_fwd", "chunk_fwd_gva", "chunk_fwd_varlen", "decode_step", "gate_prologue_bwd",
           "gate_prologue_fwd", "kv_compact", "kv_fork", "kv_reserve", "lib", "rope_freqs", "status_string",
           "workspace_bytes", "workspace_bytes_gva", "workspace_bytes_varlen"]
