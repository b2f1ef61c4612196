"""libdcpmerge: the decode-context-parallel (DCP) attention partial-merge path
for AMD Instinct MI355X (gfx950).

Hand-written HIP kernels behind a C ABI (include/dcpmerge.h) for the three
steps of the path -- the stride-driven pack of rank-local partials into
per-peer send layouts, the LSE-weighted unpack-combine, and the in-place
merge -- with a thin ctypes binding.  The shared library is loaded on first
use and every call fails loudly if it is missing.

The attention side of a rank, around that path, is in attn.py (libdcpattn.so,
include/dcpattn.h): norm, rotation and cache append of new tokens, attention
over the rank's paged cache, accumulated attention weights, and eviction.
"""
from ._lib import DcpError, DcpLaunchError
from .attn import AttnError, cache_slots, dcp_attn_mass, dcp_cache_evict, dcp_paged_attn, owned_positions, qk_norm_rope_append
from .ops import cp_lse_combine_inplace, dcp_lse_combine, dcp_pack_a2a_send, interleaved_views, lse_pack_dim

__all__ = ["AttnError", "DcpError", "DcpLaunchError", "cache_slots", "cp_lse_combine_inplace", "dcp_attn_mass",
           "dcp_cache_evict", "dcp_lse_combine", "dcp_pack_a2a_send", "dcp_paged_attn", "interleaved_views",
           "lse_pack_dim", "owned_positions", "qk_norm_rope_append"]
