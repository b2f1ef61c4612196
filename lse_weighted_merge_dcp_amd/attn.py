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
  dcp_attn_mass         accumulate the attention weight of every cached key
                        from the LSE that ops.dcp_lse_combine returns
  dcp_cache_evict       keep the keys of highest accumulated weight
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
from typing import Optional, Tuple

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
}
# The argument structs: every field 8 bytes, in the header's order.
ROPE_ARGS = struct.Struct("=45q3d")
ATTN_ARGS = struct.Struct("=41q3d")
EVICT_ARGS = struct.Struct("=33q")

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
        v_cache.data_ptr() if v_cache is not None else 0, vs[0], vs[1], vs[2],
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
    h = lib()
    args = _attn_args(q, k_cache, v_cache, block_table, cu_q, kv_len, seq_len, scale, Dv, rank, n_ranks, interleave,
                      causal, k_scale, v_scale, is_lse_base_on_e, wide_weights, out, out_lse, 0, 0)
    args, _keep = _with_workspace(args, h.dcpa_paged_attn_workspace, "dcpa_paged_attn", workspace, q)
    _call(h.dcpa_paged_attn, "dcpa_paged_attn", dev, args)
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
