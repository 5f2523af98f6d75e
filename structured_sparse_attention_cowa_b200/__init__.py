"""CoWindow Attention (CoWA) for NVIDIA B200 (sm_100a).

The compute lives in libcowa.so (hand-written CUDA: TMA + tcgen05 forward and
backward kernels, split-KV decode kernels over contiguous, compacted and paged
caches, rotary positions); `cowa` is its Python binding (ctypes, and _binding.so
for the calls of a serving step).
"""

from .cowa import (CowaError, Pattern, Rope, compact_append, compact_cache, compact_rows, cowa_bwd,  # noqa: F401
                   cowa_bwd_varlen,
                   cowa_decode, cowa_decode_compact, cowa_decode_paged, cowa_decode_paged_fp8, cowa_fwd, cowa_fwd_chunk,
                   cowa_fwd_paged, cowa_fwd_varlen, cowa_rope, cowa_rope_bwd, lib, paged_append, paged_append_fp8, pages_needed,
                   plan_debug, rope_frequencies, visible_counts, workspace_status)

__all__ = ["Pattern", "CowaError", "cowa_fwd", "cowa_fwd_chunk", "cowa_fwd_varlen", "cowa_bwd", "cowa_bwd_varlen", "cowa_decode", "cowa_decode_compact",
           "compact_rows", "compact_cache", "compact_append", "lib", "plan_debug", "visible_counts",
           "workspace_status", "Rope", "rope_frequencies", "cowa_rope", "cowa_rope_bwd", "paged_append",
           "paged_append_fp8", "cowa_decode_paged", "cowa_decode_paged_fp8", "cowa_fwd_paged", "pages_needed"]
