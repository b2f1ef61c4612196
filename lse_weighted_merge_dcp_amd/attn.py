"""Python API of libdcpattn: the attention side of a decode-context-parallel
rank, before and after the merge of ops.py.

Argument marshalling only, as in ops.py: tensors become device pointers,
element strides and sizes, packed into the argument structs of
include/dcpattn.h, and every step runs in the HIP kernels of libdcpattn.so on
the tensors' device and that device's current stream.  There is no CPU or
PyTorch fallback.

  qk_norm_rope_append   norm and rotate new queries and keys, write the rank's
                        keys and values into its paged cache
  dcp_paged_attn        attention of new tokens over the rank's cache: the
                        partial output and LSE that ops.dcp_pack_a2a_send takes
  dcp_prefix_attn       the same for a batch whose sequences share the first keys
                        of their caches, which are read once for a group
  dcp_attn_mass         accumulate the attention weight of every cached key
                        from the LSE that ops.dcp_lse_combine returns
  dcp_cache_evict       keep the keys of highest accumulated weight
  latent_queries        queries into latent space, in front of attention over
                        latent rows
  latent_values         its latent outputs to values
  latent_expand         keys and values of every head from cached latent rows
  dcp_latent_attn       attention over them: latent attention in the expanded form
  dcp_batch_plan        a step's lengths, page tables, positions and cache slots
                        from the numbers of new tokens, on the GPU
  cache_slots           where this rank caches new tokens
  owned_positions       how many positions of a sequence lie on this rank

Under DCP the token at position p lies on rank (p // interleave) % n_ranks: the
round-robin length formula of sglang PR #33926 report, 实现拆解 item 2, in
blocks of `interleave` positions.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from .ops import _on_gpu, _require, _stream

ATTN_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdcpattn.so")

STATUS = dict(_lib.STATUS)
STATUS.update({-20: "DCPA_ERR_WORKSPACE", -21: "DCPA_ERR_VALUE"})

_I64, _VP, _CP = ctypes.c_int64, ctypes.c_void_p, ctypes.c_char_p
SIGNATURES = {
    "dcpa_status_str": ([ctypes.c_int], _CP),
    "dcpa_qk_norm_rope_append": ([_CP, _VP], ctypes.c_int),
    "dcpa_paged_attn": ([_CP, _VP], ctypes.c_int),
    "dcpa_paged_attn_workspace": ([_CP], _I64),
    "dcpa_attn_mass": ([_CP, _VP, _I64, _I64, _I64, _VP], ctypes.c_int),
    "dcpa_attn_mass_workspace": ([_CP], _I64),
    "dcpa_cache_evict": ([_CP, _VP], ctypes.c_int),
    "dcpa_batch_plan": ([_CP, _VP], ctypes.c_int),
    "dcpa_prefix_attn": ([_CP, _VP, _VP, _I64, _VP], ctypes.c_int),
    "dcpa_prefix_attn_workspace": ([_CP, _I64], _I64),
    "dcpa_pair_attn": ([_CP] + [_VP, _I64, _I64, _I64, _I64] + [_VP, _I64, _I64, _I64] + [_VP], ctypes.c_int),
    "dcpa_pair_attn_workspace": ([_CP], _I64),
    "dcpa_project": ([_CP, _VP], ctypes.c_int),
    "dcpa_latent_expand": ([_CP, _VP], ctypes.c_int),
    "dcpa_latent_attn": ([_CP, _CP, _VP], ctypes.c_int),
    "dcpa_latent_attn_workspace": ([_CP, _CP], _I64),
}
# The argument structs: every field 8 bytes, in the header's order.
ROPE_ARGS = struct.Struct("=45q3d")
ATTN_ARGS = struct.Struct("=41q3d")
EVICT_ARGS = struct.Struct("=33q")
PLAN_ARGS = struct.Struct("=23q")
PROJECT_ARGS = struct.Struct("=16q")
EXPAND_ARGS = struct.Struct("=42q1d")

_DTYPE = {torch.float16: _lib.DCP_F16, torch.bfloat16: _lib.DCP_BF16}
_CACHE = {torch.float16: _lib.DCP_F16, torch.bfloat16: _lib.DCP_BF16, torch.float8_e4m3fn: _lib.DCP_FP8_E4M3}

_handle = None


def lib():
    """libdcpattn.so, loaded on first use (raises if it is not built)."""
    global _handle
    if _handle is None:
        if not os.path.exists(ATTN_LIB_PATH):
            raise ImportError("libdcpattn.so is not built (expected at %s); run "
                              "`python -m lse_weighted_merge_dcp_amd.csrc.build`" % ATTN_LIB_PATH)
        h = ctypes.CDLL(ATTN_LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = res
        _handle = h
    return _handle


class AttnError(_lib.DcpError):
    """A libdcpattn call rejected its arguments (nothing was enqueued)."""

    def __init__(self, status: int, fn: str):
        ValueError.__init__(self, "%s failed: %s" % (fn, STATUS.get(status, status)))
        self.status = status


def _check(status: int, fn: str) -> None:
    if status == -9:
        raise _lib.DcpLaunchError("%s failed: DCP_ERR_LAUNCH" % fn)
    if status != 0:
        raise AttnError(status, fn)


def _call(fn, name: str, device: int, *args) -> None:
    """fn(*args, stream) with the tensors' device current."""
    if device == torch.cuda.current_device():
        st = fn(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _stream(device))
    _check(st, name)


def _rows(t: torch.Tensor, name: str, nd: int) -> None:
    if t.dim() != nd:
        raise ValueError("%s: expected %d dimensions, got %d" % (name, nd, t.dim()))
    if not (t.stride(-1) == 1 or t.shape[-1] == 1 or t.numel() == 0):
        raise ValueError("%s: the last dimension must be contiguous" % name)


def _ints(t: torch.Tensor, name: str, shape, dtype=torch.int32) -> None:
    if t.dtype != dtype or tuple(t.shape) != shape or not (t.is_contiguous() or t.dim() == 2 and t.stride(1) == 1):
        raise ValueError("%s must be contiguous %s %s" % (name, dtype, list(shape)))


def _cache_types(dtype: torch.dtype, *caches) -> Tuple[int, int]:
    if dtype not in _DTYPE:
        raise ValueError("unsupported dtype %s (float16 or bfloat16)" % dtype)
    for c in caches:
        if c is not None and c.dtype not in (dtype, torch.float8_e4m3fn):
            raise ValueError("a cache holds the queries' type or float8_e4m3fn, not %s" % c.dtype)
        if c is not None and c.dtype != caches[0].dtype:
            raise ValueError("k_cache and v_cache must have one type")
    return _DTYPE[dtype], _CACHE[caches[0].dtype]


def qk_norm_rope_append(q: torch.Tensor, k: torch.Tensor, v: Optional[torch.Tensor], q_weight: Optional[torch.Tensor],
                        k_weight: Optional[torch.Tensor], positions: torch.Tensor, cos_sin: torch.Tensor,
                        slots: torch.Tensor, k_cache: torch.Tensor, v_cache: Optional[torch.Tensor], *,
                        rope_offset: int = 0, interleaved: bool = False, eps: float = 1e-6, k_scale: float = 1.0,
                        v_scale: float = 1.0, mass: Optional[torch.Tensor] = None,
                        q_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Norm and rotate new queries q [T,Hq,D] and keys k [T,Hkv,D], and write
    the keys and the values v [T,Hkv,Dv] (or None: the latent layout) into the
    cache rows slots [T] (int64: page * page_size + place; a slot outside the
    cache is skipped).  q_weight / k_weight [n] norm the first n columns of
    every head (None: no norm); cos_sin [P, rot] fp32 holds the cosines and
    then the sines of each position, applied to the rot columns from
    rope_offset on, to columns (j, j + rot/2), or (2j, 2j+1) if interleaved.
    positions [T] is int32.  An 8-bit cache stores value / scale, rounded to
    nearest even.  mass [pages,page_size,Hkv] (fp32, of dcp_attn_mass): the weight
    of every key that is written starts at 0, whatever an earlier key left there.
    Returns q_out [T,Hq,D] (q itself may be given)."""
    dev = _on_gpu(q, k, v, q_weight, k_weight, positions, cos_sin, slots, k_cache, v_cache, mass, q_out)
    for t, name, nd in ((q, "q", 3), (k, "k", 3), (k_cache, "k_cache", 4), (cos_sin, "cos_sin", 2)):
        _rows(t, name, nd)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    pages, page_size = k_cache.shape[0], k_cache.shape[1]
    if k.shape != (T, Hkv, D) or k_cache.shape[2:] != (Hkv, D) or k.dtype != q.dtype:
        raise ValueError("expected q [T,Hq,D], k [T,Hkv,D] of one dtype and k_cache [pages,page_size,Hkv,D]")
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    Dv, vs, vcs = 0, (0, 0), (0, 0, 0)
    if v is not None:
        _rows(v, "v", 3)
        _rows(v_cache, "v_cache", 4)
        Dv = v.shape[2]
        if v.shape[:2] != (T, Hkv) or v_cache.shape != (pages, page_size, Hkv, Dv) or v.dtype != q.dtype:
            raise ValueError("expected v [T,Hkv,Dv] and v_cache [pages,page_size,Hkv,Dv]")
        vs, vcs = v.stride(), v_cache.stride()
    dt, ct = _cache_types(q.dtype, k_cache, v_cache)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and not (w.dtype == q.dtype and w.dim() == 1 and w.is_contiguous()):
            raise ValueError("%s must be a contiguous vector of the queries' dtype" % name)
    _ints(positions, "positions", (T,))
    _ints(slots, "slots", (T,), torch.int64)
    if mass is not None and (mass.shape != k_cache.shape[:3] or mass.dtype != torch.float32):
        raise ValueError("mass must be float32 [pages,page_size,Hkv]")
    if cos_sin.dtype != torch.float32:
        raise ValueError("cos_sin is float32 [positions, rot]")
    if q_out is None:
        q_out = torch.empty((T, Hq, D), dtype=q.dtype, device=q.device)
    _rows(q_out, "q_out", 3)
    if q_out.shape != (T, Hq, D) or q_out.dtype != q.dtype:
        raise ValueError("bad q_out tensor")
    qs, ks, os_, kcs = q.stride(), k.stride(), q_out.stride(), k_cache.stride()
    ms = mass.stride() if mass is not None else (0, 0, 0)
    args = ROPE_ARGS.pack(
        q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1],
        v.data_ptr() if v is not None else 0, vs[0], vs[1],
        q_weight.data_ptr() if q_weight is not None else 0, k_weight.data_ptr() if k_weight is not None else 0,
        positions.data_ptr(), cos_sin.data_ptr(), cos_sin.stride(0), slots.data_ptr(),
        q_out.data_ptr(), os_[0], os_[1], k_cache.data_ptr(), kcs[0], kcs[1], kcs[2],
        v_cache.data_ptr() if v is not None else 0, vcs[0], vcs[1], vcs[2],
        mass.data_ptr() if mass is not None else 0, ms[0], ms[1], ms[2],
        T, Hq, Hkv, D, Dv, q_weight.shape[0] if q_weight is not None else 0,
        k_weight.shape[0] if k_weight is not None else 0, rope_offset, cos_sin.shape[1], 1 if interleaved else 0,
        cos_sin.shape[0], pages, page_size, dt, ct, eps, k_scale, v_scale)
    _call(lib().dcpa_qk_norm_rope_append, "dcpa_qk_norm_rope_append", dev, args)
    return q_out


# The address of a value cache without pages, never followed (torch has none for it; NULL says that values lie within the
# keys, which have other limits).
_NO_PAGES = 16


def _attn_args(q, k_cache, v_cache, block_table, cu_q, kv_len, seq_len, scale, Dv, rank, n_ranks, interleave, causal,
               k_scale, v_scale, base_e, wide, out, lse, ws, ws_bytes):
    """The packed dcpa_attn_args of an attention or weight call."""
    T, Hq, Dk = q.shape
    pages, page_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape[3] != Dk:
        raise ValueError("q has %d columns, k_cache %d" % (Dk, k_cache.shape[3]))
    B = kv_len.shape[0]
    _ints(kv_len, "kv_len", (B,))
    _ints(cu_q, "cu_q", (B + 1,))
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, pages of a sequence]")
    _ints(block_table, "block_table", (B, block_table.shape[1]))
    if seq_len is not None:
        _ints(seq_len, "seq_len", (B,))
    elif causal and n_ranks > 1:
        raise ValueError("seq_len is needed to order the keys of several ranks")
    dt, ct = _cache_types(q.dtype, k_cache, v_cache)
    qs, ks = q.stride(), k_cache.stride()
    vs = v_cache.stride() if v_cache is not None else (0, 0, 0)
    os_ = out.stride() if out is not None else (0, 0)
    ls = lse.stride() if lse is not None else (0, 0)
    if scale is None:
        scale = Dk ** -0.5
    return ATTN_ARGS.pack(
        q.data_ptr(), qs[0], qs[1], k_cache.data_ptr(), ks[0], ks[1], ks[2],
        (v_cache.data_ptr() or _NO_PAGES) if v_cache is not None else 0, vs[0], vs[1], vs[2],
        block_table.data_ptr(), block_table.stride(0), cu_q.data_ptr(), kv_len.data_ptr(),
        seq_len.data_ptr() if seq_len is not None else 0,
        out.data_ptr() if out is not None else 0, os_[0], os_[1],
        lse.data_ptr() if lse is not None else 0, ls[0], ls[1], ws, ws_bytes,
        B, T, Hq, Hkv, Dk, Dv, pages, page_size, block_table.shape[1],
        n_ranks, rank, interleave, 1 if causal else 0, dt, ct,
        _lib.DCP_LSE_BASE_E if base_e else _lib.DCP_LSE_BASE_2, 1 if wide else 0, scale, k_scale, v_scale)


_WS_AT = 22 * 8      # offset of workspace and workspace_bytes in the packed struct


def _with_workspace(args: bytes, query, name: str, workspace: Optional[torch.Tensor], like: torch.Tensor):
    """args with a workspace: the caller's, or a fresh allocation of the size
    the library asks for (none if it needs none)."""
    need = query(args)
    if need < 0:
        _check(need, name)
    if need == 0:
        return args, None
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the tensors' device")
    w = struct.pack("=2q", workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return args[:_WS_AT] + w + args[_WS_AT + 16:], workspace


def _attn_outputs(q, k_cache, v_cache, v_dim, out, out_lse):
    """The checked shapes of an attention call: (Dv, out, out_lse), allocated where they are not given."""
    _rows(q, "q", 3)
    _rows(k_cache, "k_cache", 4)
    T, Hq, Dk = q.shape
    if v_cache is None:
        if v_dim is None:
            raise ValueError("v_dim is needed where the values are columns of the keys")
        Dv = v_dim
    else:
        _rows(v_cache, "v_cache", 4)
        Dv = v_cache.shape[3]
        if v_cache.shape[:3] != k_cache.shape[:3] or (v_dim is not None and v_dim != Dv):
            raise ValueError("v_cache must be [pages,page_size,Hkv,Dv] beside k_cache")
    if out is None:
        out = torch.empty((T, Hq, Dv), dtype=q.dtype, device=q.device)
    if out_lse is None:
        out_lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    _rows(out, "out", 3)
    if out.shape != (T, Hq, Dv) or out.dtype != q.dtype:
        raise ValueError("bad out tensor")
    if out_lse.shape != (T, Hq) or out_lse.dtype != torch.float32:
        raise ValueError("bad out_lse tensor")
    return Dv, out, out_lse


def dcp_paged_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: Optional[torch.Tensor],
                   block_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, *,
                   seq_len: Optional[torch.Tensor] = None, scale: Optional[float] = None, v_dim: Optional[int] = None,
                   rank: int = 0, n_ranks: int = 1, interleave: int = 1, causal: bool = True, k_scale: float = 1.0,
                   v_scale: float = 1.0, is_lse_base_on_e: bool = True, wide_weights: bool = False,
                   out: Optional[torch.Tensor] = None, out_lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Attention of the new tokens q [T,Hq,Dk] over this rank's paged cache:
    k_cache [pages,page_size,Hkv,Dk], v_cache [pages,page_size,Hkv,Dv], or None
    with v_dim = Dv: values are the first Dv columns of the keys.  Sequence b's
    tokens are rows cu_q[b]..cu_q[b+1]-1 (int32 [B+1]), its cached keys the
    first kv_len[b] places of the pages block_table[b] (int32), this step's own
    keys among them; seq_len[b] is its whole length over all ranks (needed if
    causal and n_ranks > 1).  Returns (out [T,Hq,Dv], lse [T,Hq] fp32), which
    ops.dcp_pack_a2a_send takes; a token that sees no key on this rank gets the
    neutral pair (0, -inf).  Rows outside the sequences are left as they were.
    scale defaults to Dk ** -0.5.  The weights are rounded to q's type for the
    product with the values; with wide_weights what the rounding leaves takes a
    second product (1.2 to 1.4 times as long for many or latent rows; few rows
    have it always)."""
    dev = _on_gpu(q, k_cache, v_cache, block_table, cu_q, kv_len, seq_len, out, out_lse, workspace)
    Dv, out, out_lse = _attn_outputs(q, k_cache, v_cache, v_dim, out, out_lse)
    h = lib()
    args = _attn_args(q, k_cache, v_cache, block_table, cu_q, kv_len, seq_len, scale, Dv, rank, n_ranks, interleave,
                      causal, k_scale, v_scale, is_lse_base_on_e, wide_weights, out, out_lse, 0, 0)
    args, _keep = _with_workspace(args, h.dcpa_paged_attn_workspace, "dcpa_paged_attn", workspace, q)
    _call(h.dcpa_paged_attn, "dcpa_paged_attn", dev, args)
    return out, out_lse


def dcp_prefix_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: Optional[torch.Tensor],
                    block_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, cu_group: torch.Tensor,
                    shared_len: torch.Tensor, *, seq_len: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    v_dim: Optional[int] = None, rank: int = 0, n_ranks: int = 1, interleave: int = 1,
                    causal: bool = True, k_scale: float = 1.0, v_scale: float = 1.0, is_lse_base_on_e: bool = True,
                    wide_weights: bool = False, out: Optional[torch.Tensor] = None,
                    out_lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """dcp_paged_attn for a batch whose sequences share the first keys of their
    caches (a common system prompt or document): the same result, with the shared
    keys read once for all rows of a group.  Group g is the sequences
    cu_group[g]..cu_group[g+1]-1 (int32 [groups+1]); the first shared_len[g]
    (int32 [groups]) cached keys of each of them on this rank are the same: whole
    pages that stand in all their rows of block_table.  Sequences outside the
    groups share nothing.  For one or a few new tokens to a sequence; prompt chunks
    (128 rows of a key head and more to a sequence) run as in dcp_paged_attn.  Returns
    (out [T,Hq,Dv], lse [T,Hq] fp32).  Weights are rounded or not as in dcp_paged_attn
    (wide_weights)."""
    dev = _on_gpu(q, k_cache, v_cache, block_table, cu_q, kv_len, seq_len, cu_group, shared_len, out, out_lse, workspace)
    Dv, out, out_lse = _attn_outputs(q, k_cache, v_cache, v_dim, out, out_lse)
    groups = shared_len.shape[0] if shared_len.dim() == 1 else -1
    _ints(shared_len, "shared_len", (groups,))
    _ints(cu_group, "cu_group", (groups + 1,))
    h = lib()
    args = _attn_args(q, k_cache, v_cache, block_table, cu_q, kv_len, seq_len, scale, Dv, rank, n_ranks, interleave,
                      causal, k_scale, v_scale, is_lse_base_on_e, wide_weights, out, out_lse, 0, 0)
    args, _keep = _with_workspace(args, lambda a: h.dcpa_prefix_attn_workspace(a, groups), "dcpa_prefix_attn", workspace, q)
    _call(h.dcpa_prefix_attn, "dcpa_prefix_attn", dev, args, cu_group.data_ptr(), shared_len.data_ptr(), groups)
    return out, out_lse


def dcp_attn_mass(q: torch.Tensor, k_cache: torch.Tensor, lse: torch.Tensor, mass: torch.Tensor,
                  block_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, *,
                  seq_len: Optional[torch.Tensor] = None, scale: Optional[float] = None, rank: int = 0,
                  n_ranks: int = 1, interleave: int = 1, causal: bool = True, k_scale: float = 1.0,
                  is_lse_base_on_e: bool = True, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Add to mass [pages,page_size,Hkv] (fp32) the attention weight that the
    new tokens q give each cached key of this rank: the sum over the tokens and
    the heads of the key's group of exp(s - lse), lse [T,Hq] fp32 the merged
    log-sum-exp of all ranks (ops.dcp_lse_combine; a rank that merged only its
    own heads gathers the others' first).  A new key's weight has to start at 0
    (qk_norm_rope_append's mass).  The other arguments are those of
    dcp_paged_attn.  A page may stand only once in the block_table of a call.
    Returns mass."""
    dev = _on_gpu(q, k_cache, lse, mass, block_table, cu_q, kv_len, seq_len, workspace)
    _rows(q, "q", 3)
    _rows(k_cache, "k_cache", 4)
    if lse.shape != q.shape[:2] or lse.dtype != torch.float32:
        raise ValueError("lse must be float32 [T,Hq]")
    if mass.shape != k_cache.shape[:3] or mass.dtype != torch.float32:
        raise ValueError("mass must be float32 [pages,page_size,Hkv]")
    h = lib()
    args = _attn_args(q, k_cache, None, block_table, cu_q, kv_len, seq_len, scale, 8, rank, n_ranks, interleave,
                      causal, k_scale, 1.0, is_lse_base_on_e, False, None, lse, 0, 0)
    args, _keep = _with_workspace(args, h.dcpa_attn_mass_workspace, "dcpa_attn_mass", workspace, q)
    m = mass.stride()
    _call(h.dcpa_attn_mass, "dcpa_attn_mass", dev, args, mass.data_ptr(), m[0], m[1], m[2])
    return mass


def dcp_cache_evict(mass: torch.Tensor, k_cache: torch.Tensor, v_cache: Optional[torch.Tensor],
                    block_table: torch.Tensor, kv_len: torch.Tensor, dst_table: torch.Tensor, budget: int, *,
                    n_sink: int = 0, n_recent: int = 0, new_len: Optional[torch.Tensor] = None,
                    kept: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Cut each sequence's cache to `budget` keys for every key head: the first
    n_sink, the last n_recent and of the others those of highest mass
    [pages,page_size,Hkv] (ties to the oldest).  The kept keys, their values
    and their mass are copied, in their old order, into the pages
    dst_table[b] (int32 [B, pages]) of the same pools, whose other places stay as
    they are (give mass to qk_norm_rope_append); source pages are only read, and
    must not be among the destinations.  Returns (new_len [B] int32, which may be
    kv_len itself, kept [B,Hkv,budget] int32: the old index of each kept key, -1
    behind the last)."""
    dev = _on_gpu(mass, k_cache, v_cache, block_table, kv_len, dst_table, new_len, kept)
    _rows(k_cache, "k_cache", 4)
    pages, page_size, Hkv, Dk = k_cache.shape
    if mass.shape != (pages, page_size, Hkv) or mass.dtype != torch.float32:
        raise ValueError("mass must be float32 [pages,page_size,Hkv]")
    Dv, vs = 0, (0, 0, 0)
    if v_cache is not None:
        _rows(v_cache, "v_cache", 4)
        if v_cache.shape[:3] != (pages, page_size, Hkv) or v_cache.dtype != k_cache.dtype:
            raise ValueError("v_cache must be [pages,page_size,Hkv,Dv] beside k_cache, of one type")
        Dv, vs = v_cache.shape[3], v_cache.stride()
    B = kv_len.shape[0]
    _ints(kv_len, "kv_len", (B,))
    for t, name in ((block_table, "block_table"), (dst_table, "dst_table")):
        if t.dim() != 2:
            raise ValueError("%s must be int32 [B, pages of a sequence]" % name)
        _ints(t, name, (B, t.shape[1]))
    _require(budget >= 0, "budget must not be negative")
    if new_len is None:
        new_len = torch.empty(B, dtype=torch.int32, device=mass.device)
    if kept is None:
        kept = torch.empty((B, Hkv, budget), dtype=torch.int32, device=mass.device)
    _ints(new_len, "new_len", (B,))
    _rows(kept, "kept", 3)
    if kept.shape != (B, Hkv, budget) or kept.dtype != torch.int32:
        raise ValueError("kept must be int32 [B,Hkv,budget]")
    m, ks, kp = mass.stride(), k_cache.stride(), kept.stride()
    args = EVICT_ARGS.pack(
        mass.data_ptr(), m[0], m[1], m[2], k_cache.data_ptr(), ks[0], ks[1], ks[2],
        v_cache.data_ptr() if v_cache is not None else 0, vs[0], vs[1], vs[2],
        block_table.data_ptr(), block_table.stride(0), kv_len.data_ptr(), dst_table.data_ptr(), dst_table.stride(0),
        new_len.data_ptr(), kept.data_ptr(), kp[0], kp[1],
        B, Hkv, Dk, Dv, k_cache.element_size(), pages, page_size, block_table.shape[1], dst_table.shape[1],
        budget, n_sink, n_recent)
    _call(lib().dcpa_cache_evict, "dcpa_cache_evict", dev, args)
    return new_len, kept


def _project(x, w, turned, N, K, copy, out, name):
    """One dcpa_project call: w [H, ., .] with its rows as columns of the result (turned: as sums)."""
    dev = _on_gpu(x, w, out)
    _rows(x, "x", 3)
    T, H = x.shape[0], x.shape[1]
    if x.dtype not in _DTYPE or w.dtype != x.dtype:
        raise ValueError("%s: float16 or bfloat16 rows and weights of one dtype" % name)
    if out is None:
        out = torch.empty((T, H, N + copy), dtype=x.dtype, device=x.device)
    _rows(out, "out", 3)
    if out.shape != (T, H, N + copy) or out.dtype != x.dtype:
        raise ValueError("bad out tensor")
    if out.numel() > 0 and out.data_ptr() in (x.data_ptr(), w.data_ptr()):
        raise ValueError("%s: out must not lie over its inputs" % name)
    xs, ws, ys = x.stride(), w.stride(), out.stride()
    w_N, w_K = (ws[2], ws[1]) if turned else (ws[1], ws[2])
    args = PROJECT_ARGS.pack(x.data_ptr(), xs[0], xs[1], w.data_ptr(), ws[0], w_N, w_K, out.data_ptr(), ys[0], ys[1],
                             T, H, N, K, copy, _DTYPE[x.dtype])
    _call(lib().dcpa_project, "dcpa_project", dev, args)
    return out


def latent_queries(q: torch.Tensor, w_uk: torch.Tensor, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Queries q [T,H,Dn+Dr] into latent space: [q[..., :Dn] @ w_uk[h] | q[...,
    Dn:]], [T,H,Dc+Dr], with the key weights w_uk [H,Dn,Dc] of a latent layer.
    The result is what qk_norm_rope_append (rope_offset = Dc) and dcp_paged_attn
    take against latent rows.  w_uk may be a view of the whole projection
    [H,Dn+Dv,Dc], or of a transposed one (one of its last two dimensions
    contiguous).  out must not lie over q or w_uk."""
    if w_uk.dim() != 3 or q.dim() != 3 or w_uk.shape[0] != q.shape[1] or q.shape[2] < w_uk.shape[1]:
        raise ValueError("expected q [T,H,Dn+Dr] and w_uk [H,Dn,Dc]")
    Dn, Dc = w_uk.shape[1], w_uk.shape[2]
    return _project(q, w_uk, True, Dc, Dn, q.shape[2] - Dn, out, "latent_queries")


def latent_values(o: torch.Tensor, w_uv: torch.Tensor, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Values [T,H,Dv] from (merged) latent outputs o [T,H,Dc]: o[t, h] @
    w_uv[h].T, with the value weights w_uv [H,Dv,Dc] of a latent layer (one of
    the last two dimensions contiguous).  out must not lie over o or w_uv."""
    if w_uv.dim() != 3 or o.dim() != 3 or w_uv.shape[0] != o.shape[1] or o.shape[2] != w_uv.shape[2]:
        raise ValueError("expected o [T,H,Dc] and w_uv [H,Dv,Dc]")
    return _project(o, w_uv, False, w_uv.shape[1], w_uv.shape[2], 0, out, "latent_values")


def _expand_args(kv_cache, w_uk, w_uv, block_table, kv_len, max_keys, k_scale, k_out, v_out, k_rest, v_rest, places):
    """The packed dcpa_expand_args of an expansion, and its outputs, allocated where they are not given."""
    for t, name, nd in ((kv_cache, "kv_cache", 4), (w_uk, "w_uk", 3), (w_uv, "w_uv", 3)):
        _rows(t, name, nd)
    H, Dn, Dc = w_uk.shape
    Dv, Dr = w_uv.shape[1], kv_cache.shape[3] - Dc
    if w_uv.shape != (H, Dv, Dc) or w_uv.dtype != w_uk.dtype or kv_cache.shape[2] != 1 or Dr < 0:
        raise ValueError("expected kv_cache [pages,page_size,1,Dc+Dr], w_uk [H,Dn,Dc] and w_uv [H,Dv,Dc] of one dtype")
    dt, ct = _cache_types(w_uk.dtype, kv_cache)
    B = kv_len.shape[0]
    _ints(kv_len, "kv_len", (B,))
    if block_table.dim() != 2:
        raise ValueError("block_table must be int32 [B, pages of a sequence]")
    _ints(block_table, "block_table", (B, block_table.shape[1]))
    _require(max_keys >= 0, "max_keys must not be negative")
    if (k_rest is None) != (v_rest is None):
        raise ValueError("k_rest and v_rest go together")
    if k_out is None:
        k_out = torch.empty((B, max_keys, H, Dn + Dr), dtype=w_uk.dtype, device=w_uk.device)
    if v_out is None:
        v_out = torch.empty((B, max_keys, H, Dv), dtype=w_uk.dtype, device=w_uk.device)
    strides = []
    for t, name, d in ((k_out, "k_out", Dn + Dr), (v_out, "v_out", Dv), (k_rest, "k_rest", Dn), (v_rest, "v_rest", Dv)):
        if t is None:
            strides += [0, 0, 0, 0]
            continue
        _rows(t, name, 4)
        if t.shape != (B, max_keys, H, d) or t.dtype != w_uk.dtype:
            raise ValueError("%s must be [B,max_keys,H,%d] of the weights' dtype" % (name, d))
        strides += [t.data_ptr(), *t.stride()[:3]]
    if places is not None:
        _ints(places, "places", (B, max_keys))
    cs, wk, wv = kv_cache.stride(), w_uk.stride(), w_uv.stride()
    return EXPAND_ARGS.pack(
        kv_cache.data_ptr(), cs[0], cs[1], block_table.data_ptr(), block_table.stride(0), kv_len.data_ptr(),
        w_uk.data_ptr(), wk[0], wk[1], w_uv.data_ptr(), wv[0], wv[1], *strides,
        places.data_ptr() if places is not None else 0, places.stride(0) if places is not None else 0,
        B, H, Dn, Dr, Dv, Dc, max_keys, kv_cache.shape[0], kv_cache.shape[1], block_table.shape[1], dt, ct, k_scale), k_out, v_out


def latent_expand(kv_cache: torch.Tensor, w_uk: torch.Tensor, w_uv: torch.Tensor, block_table: torch.Tensor,
                  kv_len: torch.Tensor, max_keys: int, *, k_scale: float = 1.0, k_out: Optional[torch.Tensor] = None,
                  v_out: Optional[torch.Tensor] = None, k_rest: Optional[torch.Tensor] = None,
                  v_rest: Optional[torch.Tensor] = None, places: Optional[torch.Tensor] = None):
    """Keys and values of every head from cached latent rows kv_cache
    [pages,page_size,1,Dc+Dr]: for the first kv_len[b] cached keys of each
    sequence (at most max_keys), k [B,max_keys,H,Dn+Dr] = [w_uk[h] c | rope] and
    v [B,max_keys,H,Dv] = w_uv[h] c, with w_uk [H,Dn,Dc] and w_uv [H,Dv,Dc]
    (contiguous over Dc), rounded to the weights' type.  k_rest [B,max_keys,H,Dn]
    and v_rest [B,max_keys,H,Dv] (both or neither) get what the rounding leaves, in
    the same type.  Rows behind kv_len and keys without a page are left as they
    were.  places (int32 [B,max_keys]) gets the block_table for caches of one key to a
    page, as which dcp_paged_attn takes k and v (dcp_latent_attn does it all).
    Returns (k, v)."""
    dev = _on_gpu(kv_cache, w_uk, w_uv, block_table, kv_len, k_out, v_out, k_rest, v_rest, places)
    args, k_out, v_out = _expand_args(kv_cache, w_uk, w_uv, block_table, kv_len, max_keys, k_scale, k_out, v_out, k_rest,
                                      v_rest, places)
    _call(lib().dcpa_latent_expand, "dcpa_latent_expand", dev, args)
    return k_out, v_out


def dcp_latent_attn(q: torch.Tensor, kv_cache: torch.Tensor, w_uk: torch.Tensor, w_uv: torch.Tensor,
                    block_table: torch.Tensor, cu_q: torch.Tensor, kv_len: torch.Tensor, max_keys: int, *,
                    seq_len: Optional[torch.Tensor] = None, scale: Optional[float] = None, rank: int = 0,
                    n_ranks: int = 1, interleave: int = 1, causal: bool = True, k_scale: float = 1.0,
                    is_lse_base_on_e: bool = True, wide_weights: bool = False, rounded: bool = False,
                    out: Optional[torch.Tensor] = None, out_lse: Optional[torch.Tensor] = None,
                    k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                    k_rest: Optional[torch.Tensor] = None, v_rest: Optional[torch.Tensor] = None,
                    places: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Latent attention in the expanded form: keys and values of every head are
    made from the rank's cached latent rows (latent_expand), and the new tokens'
    queries q [T,H,Dn+Dr], as the model has them (rotated, not taken into latent
    space), attend to those.  For prompt chunks: a pair of query and key costs
    Dn + Dr + Dv products (here 2 Dn + Dr + 2 Dv) instead of the latent form's 2 Dc +
    Dr, a key H (Dn + Dv) Dc more.  Keys and values are kept in two parts, so that
    they are not rounded to 16 bits on the way; rounded=True does round them, once,
    as a cache would hold them, and is faster.  max_keys: as many keys as a sequence
    may have cached here at most; kv_len is clamped to it.  k_out, v_out, k_rest,
    v_rest (contiguous, as latent_expand has them) and places are buffers to keep
    them in, fresh ones if not given; they hold keys and values divided by what is left
    of k_scale without a power of two (dcpa_latent_attn in the header), so that they
    are in the type's range where the keys themselves are.  The other arguments are
    those of dcp_paged_attn.  Returns (out [T,H,Dv], lse [T,H])."""
    B, (H, Dn, _), Dv = kv_len.shape[0], w_uk.shape, w_uv.shape[1]
    Dk = Dn + kv_cache.shape[3] - w_uk.shape[2]
    for t, name in ((k_out, "k_out"), (v_out, "v_out"), (k_rest, "k_rest"), (v_rest, "v_rest"), (places, "places")):
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    if q.dim() != 3 or q.shape[1:] != (H, Dk) or q.dtype != w_uk.dtype:
        raise ValueError("expected q [T,H,Dn+Dr] of the weights' dtype")
    if rounded and (k_rest is not None or v_rest is not None):
        raise ValueError("rounded keys and values have no rest")
    # (one call, whose checks are all made before it writes anything)
    dev = _on_gpu(q, kv_cache, w_uk, w_uv, block_table, cu_q, kv_len, seq_len, k_out, v_out, k_rest, v_rest, places, out,
                  out_lse, workspace)
    _require(max_keys >= 0, "max_keys must not be negative")
    if places is None:
        places = torch.empty((B, max_keys), dtype=torch.int32, device=q.device)
    if not rounded:
        if k_rest is None:
            k_rest = torch.empty((B, max_keys, H, Dn), dtype=q.dtype, device=q.device)
        if v_rest is None:
            v_rest = torch.empty((B, max_keys, H, Dv), dtype=q.dtype, device=q.device)
    make, k, v = _expand_args(kv_cache, w_uk, w_uv, block_table, kv_len, max_keys, k_scale, k_out, v_out, k_rest, v_rest,
                              places)
    k, v = k.view(B * max_keys, 1, H, Dk), v.view(B * max_keys, 1, H, Dv)
    Dv, out, out_lse = _attn_outputs(q, k, v, None, out, out_lse)
    h = lib()
    args = _attn_args(q, k, v, places, cu_q, kv_len, seq_len, scale, Dv, rank, n_ranks, interleave, causal, k_scale,
                      k_scale, is_lse_base_on_e, wide_weights, out, out_lse, 0, 0)
    args, _keep = _with_workspace(args, lambda a: h.dcpa_latent_attn_workspace(make, a), "dcpa_latent_attn", workspace, q)
    _call(h.dcpa_latent_attn, "dcpa_latent_attn", dev, make, args)
    return out, out_lse


class BatchPlan(NamedTuple):
    """What dcp_batch_plan gives a step: int32 but for slots (int64)."""
    cu_q: torch.Tensor          # [B + 1]
    seq_len: torch.Tensor       # [B], after the step
    kv_len: torch.Tensor        # [B], after the step
    free_count: torch.Tensor    # [1]
    positions: torch.Tensor     # [T]
    sequence: torch.Tensor      # [T]
    slots: torch.Tensor         # [T]


def dcp_batch_plan(new_len: torch.Tensor, seq_len: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor,
                   free_pages: torch.Tensor, free_count: torch.Tensor, max_tokens: int, page_size: int, *,
                   rank: int = 0, n_ranks: int = 1, interleave: int = 1, keep_pages: Optional[torch.Tensor] = None,
                   out: Optional[BatchPlan] = None) -> BatchPlan:
    """Plan a step with new_len[b] new tokens of sequence b (int32 [B]; negative:
    the sequence has ended), whose lengths before it are seq_len (over all ranks)
    and kv_len (cached on this rank).  Sequences that grow past their last page
    get pages from the end of free_pages (int32, of which the first
    free_count[0] are free; -1 once there are none), written into
    block_table (int32 [B, pages]); ended ones first give theirs back, but for
    the first keep_pages[b].  Returns the plan of max_tokens rows: cu_q,
    lengths after the step and pages left (negative: so many were missing), and
    for every row its position, its sequence and its slot for
    qk_norm_rope_append, -1 behind the last token (slots also where another
    rank owns the position, or no page is there).  Tokens beyond the last row
    are not taken.  out: the tensors to write; its seq_len, kv_len and free_count
    may be the inputs themselves."""
    _require(max_tokens >= 0 and page_size >= 1, "max_tokens is not negative, page_size positive")
    if new_len.dim() != 1 or block_table.dim() != 2:
        raise ValueError("new_len must be int32 [B], block_table int32 [B, pages of a sequence]")
    B, T = new_len.shape[0], max_tokens
    if out is None:
        # (one allocation: seven would take longer than the kernel)
        words = torch.empty(2 * T + (3 * B + 3) // 2, dtype=torch.int64, device=new_len.device)
        slots, rest = words.split([T, words.shape[0] - T])
        cu, seq, kv, left, pos, sid, _ = rest.view(torch.int32).split([B + 1, B, B, 1, T, T, 2 * rest.shape[0] - 3 * B - 2 - 2 * T])
        out = BatchPlan(cu, seq, kv, left, pos, sid, slots)
        dev = _on_gpu(new_len, seq_len, kv_len, block_table, free_pages, free_count, keep_pages)
    else:
        dev = _on_gpu(new_len, seq_len, kv_len, block_table, free_pages, free_count, keep_pages, *out)
        for t, name, n in ((out.cu_q, "out.cu_q", B + 1), (out.seq_len, "out.seq_len", B), (out.kv_len, "out.kv_len", B),
                           (out.free_count, "out.free_count", 1), (out.positions, "out.positions", T),
                           (out.sequence, "out.sequence", T)):
            _ints(t, name, (n,))
        _ints(out.slots, "out.slots", (T,), torch.int64)
    _ints(new_len, "new_len", (B,))
    _ints(seq_len, "seq_len", (B,))
    _ints(kv_len, "kv_len", (B,))
    if keep_pages is not None:
        _ints(keep_pages, "keep_pages", (B,))
    _ints(block_table, "block_table", (B, block_table.shape[1]))
    _ints(free_pages, "free_pages", (free_pages.numel(),))
    _ints(free_count, "free_count", (1,))
    args = PLAN_ARGS.pack(
        new_len.data_ptr(), seq_len.data_ptr(), kv_len.data_ptr(), keep_pages.data_ptr() if keep_pages is not None else 0,
        block_table.data_ptr(), block_table.stride(0) if B > 1 else block_table.shape[1], free_pages.data_ptr(),
        free_count.data_ptr(), out.free_count.data_ptr(), out.seq_len.data_ptr(), out.kv_len.data_ptr(),
        out.cu_q.data_ptr(), out.positions.data_ptr(), out.sequence.data_ptr(), out.slots.data_ptr(),
        B, max_tokens, block_table.shape[1], page_size, free_pages.numel(), n_ranks, rank, interleave)
    _call(lib().dcpa_batch_plan, "dcpa_batch_plan", dev, args)
    return out


def owned_positions(length, rank: int = 0, n_ranks: int = 1, interleave: int = 1):
    """How many of the positions 0 .. length-1 lie on this rank (length: an int
    or an integer tensor): the cached length of a sequence that has not been cut,
    and by its growth what a step adds to any."""
    block = n_ranks * interleave
    rest = length % block - rank * interleave
    rest = rest.clamp(0, interleave) if isinstance(rest, torch.Tensor) else min(max(rest, 0), interleave)
    return length // block * interleave + rest


def cache_slots(positions: torch.Tensor, sequence: torch.Tensor, block_table: torch.Tensor, page_size: int,
                rank: int = 0, n_ranks: int = 1, interleave: int = 1, *, kv_len: Optional[torch.Tensor] = None,
                seq_len: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The slots [T] (int64) that qk_norm_rope_append takes: token t of sequence
    sequence[t] at position positions[t] goes to place j % page_size of page
    block_table[sequence, j // page_size], j its index among this rank's
    positions; -1 where another rank owns it or the table has no page, and for
    padding (a negative position, or a sequence that the table has not).  Where
    caches have been cut (dcp_cache_evict), kv_len and seq_len [B] give the rank's
    cached length and the whole length of every sequence at one moment since then,
    before this step or after it alike: places count on from what is cached.
    Index arithmetic on small tensors (any device)."""
    if (kv_len is None) != (seq_len is None):
        raise ValueError("kv_len and seq_len go together")
    _require(page_size >= 1 and n_ranks >= 1 and interleave >= 1 and 0 <= rank < n_ranks,
             "page_size, n_ranks and interleave are positive, rank below n_ranks")
    rows, width = block_table.shape
    if positions.shape != sequence.shape or kv_len is not None and not kv_len.shape == seq_len.shape == (rows,):
        raise ValueError("expected positions and sequence of one shape, kv_len and seq_len [B]")
    p, s = positions.long(), sequence.long()
    if rows == 0 or width == 0:
        return torch.full_like(p, -1)
    at_row = s.clamp(0, rows - 1)
    j = owned_positions(p, rank, n_ranks, interleave)
    if kv_len is not None:
        j = j + (kv_len.long() - owned_positions(seq_len.long(), rank, n_ranks, interleave))[at_row]
    at = j // page_size
    page = block_table[at_row, at.clamp(0, width - 1)].long()
    mine = (p >= 0) & (s >= 0) & (s < rows) & (p // interleave % n_ranks == rank) & (j >= 0) & (at < width) & (page >= 0)
    return torch.where(mine, page * page_size + j % page_size, -1)
