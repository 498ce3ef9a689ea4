"""Operators around attention over libgsr: head norms with the position rotation and their gradient,
rotated cache writes, a cache of 4 bits and attention over it, verification of drafted tokens.  Argument
checks and marshalling only; include/gsr.h has the full contract of each entry point."""
from __future__ import annotations

import ctypes
import struct
from types import SimpleNamespace
from typing import NamedTuple

import torch

from .binding import GsrError, Status, lib
from .llm import _call, _dtype_code, _scratch, _Tensor, _TreeDesc, _vector


class _RopeDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("heads_q", ctypes.c_int64), ("heads_kv", ctypes.c_int64), ("seq", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("rotary_dim", ctypes.c_int64), ("table_rows", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("eps", ctypes.c_float),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
                ("positions", ctypes.c_void_p)]


class _Cache4(ctypes.Structure):
    _fields_ = [("codes", _Tensor), ("params", _Tensor)]


class _VerifyDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("total_q", ctypes.c_int64), ("vocab", ctypes.c_int64), ("max_nodes", ctypes.c_int64),
                ("target_stride_row", ctypes.c_int64), ("draft_stride_row", ctypes.c_int64)]


class Cache4(NamedTuple):
    """Keys or values in 4 bits: codes (pages, page_size, heads, D / 2) uint8 and params (pages, page_size,
    heads, D / 64, 2) float16 or bfloat16, (scale, minimum) of each 64 values; any strides."""
    codes: torch.Tensor
    params: torch.Tensor


def _declare(L) -> None:
    """Argument types of the entry points this module calls."""
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    ts, rd, c4 = ctypes.POINTER(_Tensor), ctypes.POINTER(_RopeDesc), ctypes.POINTER(_Cache4)
    L.qk_norm_rope_fwd.restype = i32
    L.qk_norm_rope_fwd.argtypes = [rd] + [ts] * 4 + [vp]
    L.qk_norm_rope_bwd_workspace.restype = i64
    L.qk_norm_rope_bwd_workspace.argtypes = [rd]
    L.qk_norm_rope_bwd.restype = i32
    L.qk_norm_rope_bwd.argtypes = [rd] + [ts] * 6 + [vp] * 3 + [i64, vp]
    L.kv_cache_append_rope.restype = i32
    L.kv_cache_append_rope.argtypes = [rd, ts, ts, ts, vp, ts, ts, ts, i64, i64, vp]
    L.kv_cache4_append_rope.restype = i32
    L.kv_cache4_append_rope.argtypes = [rd, ts, ts, ts, vp, ts, c4, c4, i64, i64, vp]
    L.kv_cache4_read.restype = i32
    L.kv_cache4_read.argtypes = [c4, c4, vp, ts, ts] + [i64] * 5 + [ctypes.c_int32, vp]
    L.tree_attention4_fwd.restype = i32
    L.tree_attention4_fwd.argtypes = [ctypes.POINTER(_TreeDesc), vp, c4, c4] + [vp] * 6 + [i64, vp]
    L.tree_attention4_workspace.restype = i64
    L.tree_attention4_workspace.argtypes = [ctypes.POINTER(_TreeDesc)]
    L.verify_drafts.restype = i32
    L.verify_drafts.argtypes = [ctypes.POINTER(_VerifyDesc)] + [vp] * 11


# The structures as bytes, for calls: a small call waits for its marshalling, and packing takes half of the time that
# making a ctypes.Structure does (norm and rotation of two operands 7.9 us, 10.6 with structures; 2.6 of them the launch).
_pack_tensor = struct.Struct("@P3q").pack
_pack_cache4 = struct.Struct("@P3qP3q").pack
_pack_rope = struct.Struct("@7q2if4P").pack
_pack_tree = struct.Struct("@13qi2fP").pack
_pack_verify = struct.Struct("@6q").pack
_entry = None


def _entries():
    """The entry points, taking addresses or bytes for every pointer."""
    global _entry
    if _entry is None:
        L, made = lib(), SimpleNamespace()
        for name in ("qk_norm_rope_fwd", "qk_norm_rope_bwd_workspace", "qk_norm_rope_bwd", "kv_cache_append_rope", "kv_cache4_append_rope",
                     "kv_cache4_read", "tree_attention4_fwd", "tree_attention4_workspace", "verify_drafts"):
            declared, function = getattr(L, name), L[name]          # a second object of the same function
            function.restype = declared.restype
            function.argtypes = [t if t in (ctypes.c_int64, ctypes.c_int32) else ctypes.c_void_p for t in declared.argtypes]
            setattr(made, name, function)
        _entry = made
    return _entry


def _call_scratch(index, stream, name, function, size_of, workspace, d, *args):
    """function(d, *args, workspace, its bytes, stream).  Without the caller's workspace the library keeps one for the
    stream, which it refuses to do in a capture: only then is there one to be made from the graph's memory."""
    if workspace is None:
        try:
            _call(index, stream, name, function, d, *args, None, 0)
            return
        except GsrError as e:
            if e.status != Status.ERR_INVALID_ARG or size_of(d) <= 0:
                raise
            ws, scratch, size = _scratch(None, lambda: size_of(d), index, stream)
            if scratch is None:
                raise
    else:
        ws, scratch, size = _scratch(workspace, None, index, stream)
    _call(index, stream, name, function, d, *args, scratch, size)


def rope_table(rows: int, rotary_dim: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """(rows, rotary_dim) float32 for ``cos_sin``: position p's cosines of p theta^(-2 i / rotary_dim), then
    their sines, computed in 64 bits (a far position's angle has too few digits in 32)."""
    freq = theta ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _rope_desc(B, Hq, Hkv, S, D, dtype, code, index, cos_sin, positions, q_weight, k_weight, eps, interleaved):
    R = rows = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be (positions, rotary_dim), got %s" % (tuple(cos_sin.shape),))
        rows, R = cos_sin.shape
    return _pack_rope(B, Hq, Hkv, S, D, R, rows, code, 1 if interleaved else 0, eps,
                      _vector(q_weight, "q_weight", D, dtype, index) or 0, _vector(k_weight, "k_weight", D, dtype, index) or 0,
                      _vector(cos_sin, "cos_sin", rows * R, torch.float32, index) or 0,
                      _vector(positions, "positions", B * S, torch.int32, index) or 0)


def _qk_desc(Q, K, cos_sin, positions, q_weight, k_weight, eps, interleaved):
    """The C description, Q's and K's shapes (K's without heads where K is None), the type and the device."""
    code, index = _dtype_code(Q, "Q"), Q.get_device()
    if index < 0:
        raise ValueError("Q must be a CUDA tensor")
    if Q.dim() != 4:
        raise ValueError("Q must be 4-D (batch, heads, seq, head_dim)")
    qs = Q.shape
    B, Hq, S, D = qs
    if K is None:
        Hkv = 0
    elif K.dim() != 4:
        raise ValueError("K must be 4-D (batch, heads, seq, head_dim)")
    else:
        Hkv = K.shape[1]
    d = _rope_desc(B, Hq, Hkv, S, D, Q.dtype, code, index, cos_sin, positions, q_weight, k_weight, eps, interleaved)
    return d, qs, (B, Hkv, S, D), Q.dtype, index


def _operand(t, name, shape, dtype, index, pages=False):
    """The C view of a 4-D operand (batch, head, row, D) of the given shape, or a cache (page, row, head, D); or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be %s on cuda:%d, got %s on %s" % (name, dtype, index, t.dtype, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    batch, head, row, one = t.stride()
    if one != 1 and shape[3] > 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return _pack_tensor(t.data_ptr(), batch, row, head) if pages else _pack_tensor(t.data_ptr(), batch, head, row)


def qk_norm_rope_fwd(Q, K, Q_out, K_out, cos_sin=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False, stream=None):
    """Norm of each head's rows and position rotation in one pass; returns Q_out, K_out.

    Q, Q_out (B, Hq, S, D), K, K_out (B, Hkv, S, D) (or both None): float16 or bfloat16, D 64 or 128 and
    contiguous, the other strides free (multiples of 8); an output may be its input.  ``q_weight``,
    ``k_weight`` (D,) of the same type: rows are normalised, y = x w / sqrt(mean(x^2) + eps); None: they are
    not.  ``cos_sin`` (positions, R) float32 (see rope_table): the first R columns are rotated, pairs (i,
    i + R / 2), or (2 i, 2 i + 1) with ``interleaved``; None: no rotation.  ``positions`` (B, S) int32 (None:
    the row's index); negative: padding, whose rows become 0.
    """
    d, qs, ks, dt, dev = _qk_desc(Q, K, cos_sin, positions, q_weight, k_weight, eps, interleaved)
    if (K is None) != (K_out is None):
        raise ValueError("K and K_out go together")
    _call(dev, stream, "qk_norm_rope_fwd", _entries().qk_norm_rope_fwd, d, _operand(Q, "Q", qs, dt, dev), _operand(K, "K", ks, dt, dev),
          _operand(Q_out, "Q_out", qs, dt, dev), _operand(K_out, "K_out", ks, dt, dev))
    return Q_out, K_out


def qk_norm_rope_bwd(dQ_out, dK_out, Q, K, dQ, dK, cos_sin=None, positions=None, q_weight=None, k_weight=None,
                     dq_weight=None, dk_weight=None, eps: float = 1e-6, interleaved: bool = False, workspace=None, stream=None):
    """Gradients dQ, dK, dq_weight, dk_weight (returned) of qk_norm_rope_fwd from those of its outputs and its inputs.

    dq_weight, dk_weight: (D,) float32, where there are weights.  dQ may be dQ_out or Q, dK likewise.
    ``workspace``: optional device buffer of qk_norm_rope_bwd_workspace(...) bytes; without one the library
    keeps one for the stream, and a call inside torch.cuda.graph takes one from the graph's memory.
    """
    d, qs, ks, dt, dev = _qk_desc(Q, K, cos_sin, positions, q_weight, k_weight, eps, interleaved)
    if not (K is None) == (dK is None) == (dK_out is None):
        raise ValueError("K, dK_out and dK go together")
    L, D, f32 = _entries(), qs[3], torch.float32
    _call_scratch(dev, stream, "qk_norm_rope_bwd", L.qk_norm_rope_bwd, L.qk_norm_rope_bwd_workspace, workspace, d, _operand(dQ_out, "dQ_out", qs, dt, dev),
          _operand(dK_out, "dK_out", ks, dt, dev), _operand(Q, "Q", qs, dt, dev), _operand(K, "K", ks, dt, dev),
          _operand(dQ, "dQ", qs, dt, dev), _operand(dK, "dK", ks, dt, dev), _vector(dq_weight, "dq_weight", D, f32, dev),
          _vector(dk_weight, "dk_weight", D, f32, dev))
    return dQ, dK, dq_weight, dk_weight


def qk_norm_rope_bwd_workspace(B: int, Hq: int, Hkv: int, S: int, D: int) -> int:
    """Bytes of workspace a qk_norm_rope_bwd call of these sizes needs."""
    n = lib().qk_norm_rope_bwd_workspace(_RopeDesc(B, Hq, Hkv, S, D))
    if n < 0:
        raise GsrError(Status.ERR_INVALID_ARG, "qk_norm_rope_bwd_workspace")
    return n


def kv_cache4(pages: int, page_size: int, heads: int, head_dim: int, dtype=torch.bfloat16, device="cuda") -> Cache4:
    """An empty cache of 4 bits, a head's rows of a page together in memory."""
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128, got %d" % head_dim)
    codes = torch.zeros(pages, heads, page_size, head_dim // 2, dtype=torch.uint8, device=device)
    params = torch.zeros(pages, heads, page_size, head_dim // 64, 2, dtype=dtype, device=device)
    return Cache4(codes.transpose(1, 2), params.transpose(1, 2))


def _cache4(c, name, shape, dtype, index):
    """The C view of a cache of 4 bits whose rows have the given (pages, page_size, heads, D)."""
    codes, params = c
    pages, page, heads, D = shape
    if codes.dtype is not torch.uint8 or params.dtype is not dtype or codes.get_device() != index or params.get_device() != index:
        raise ValueError("%s must be uint8 codes and %s params on cuda:%d, got %s, %s on %s"
                         % (name, dtype, index, codes.dtype, params.dtype, codes.device))
    if codes.shape != (pages, page, heads, D // 2) or params.shape != (pages, page, heads, D // 64, 2):
        raise ValueError("%s must have codes (%d, %d, %d, %d) and params (.., %d, 2), got %s and %s"
                         % (name, pages, page, heads, D // 2, D // 64, tuple(codes.shape), tuple(params.shape)))
    (cp, cr, ch, c1), (pp, pr, ph, pg, p1) = codes.stride(), params.stride()
    if c1 != 1 or p1 != 1 or (pg != 2 and D > 64):
        raise ValueError("%s: a row's codes, and its params, must be contiguous" % name)
    return _pack_cache4(codes.data_ptr(), cp, ch, cr, params.data_ptr(), pp, ph, pr)


def _rows(t, name, shape, dtype, index):
    """The C view of rows (tokens, heads, D)."""
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be %s on cuda:%d, got %s on %s" % (name, dtype, index, t.dtype, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    row, head, one = t.stride()
    if one != 1 and shape[2] > 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return _pack_tensor(t.data_ptr(), 0, head, row)


def _append_args(K, V, slots, Q, Q_out, cos_sin, positions, q_weight, k_weight, eps, interleaved, D, heads):
    code, index, dt = _dtype_code(K, "K"), K.get_device(), K.dtype
    if index < 0 or K.dim() != 3:
        raise ValueError("K must be a 3-D CUDA tensor (tokens, heads, head_dim)")
    N = K.shape[0]
    if (Q is None) != (Q_out is None):
        raise ValueError("Q and Q_out go together")
    Hq = 0
    if Q is not None:
        if Q.dim() != 3:
            raise ValueError("Q must be 3-D (tokens, heads, head_dim)")
        Hq = Q.shape[1]
    kv, qs = (N, heads, D), (N, Hq, D)
    d = _rope_desc(1, Hq, heads, N, D, dt, code, index, cos_sin, positions, q_weight, k_weight, eps, interleaved)
    rows = (None if Q is None else _rows(Q, "Q", qs, dt, index), _rows(K, "K", kv, dt, index), _rows(V, "V", kv, dt, index),
            _vector(slots, "slots", N, torch.int32, index), None if Q is None else _rows(Q_out, "Q_out", qs, dt, index))
    return d, rows, dt, index


def kv_cache_append_rope(K, V, slots, k_cache, v_cache, positions=None, cos_sin=None, Q=None, Q_out=None, q_weight=None,
                         k_weight=None, eps: float = 1e-6, interleaved: bool = False, stream=None):
    """kv_cache_append with K's norm and rotation on the way, and Q's into Q_out (N, Hq, D) where Q is given.

    K, V (N, H, D), slots (N,) int32 (negative: skipped), caches (pages, page_size, H, D); positions (N,) int32
    (negative: padding): kv_block_tables' for prompts, chains and single tokens, the tokens before the tree + a
    node's depth for trees.  ``cos_sin``, weights, ``eps`` and ``interleaved`` as in qk_norm_rope_fwd; Q_out may be Q.
    """
    cache = k_cache.shape
    if len(cache) != 4:
        raise ValueError("k_cache must be (pages, page_size, heads, head_dim), got %s" % (tuple(cache),))
    d, rows, dt, dev = _append_args(K, V, slots, Q, Q_out, cos_sin, positions, q_weight, k_weight, eps, interleaved, cache[3], cache[2])
    _call(dev, stream, "kv_cache_append_rope", _entries().kv_cache_append_rope, d, *rows, _operand(k_cache, "k_cache", cache, dt, dev, True),
          _operand(v_cache, "v_cache", cache, dt, dev, True), cache[0], cache[1])


def kv_cache4_append_rope(K, V, slots, k_cache, v_cache, positions=None, cos_sin=None, Q=None, Q_out=None, q_weight=None,
                          k_weight=None, eps: float = 1e-6, interleaved: bool = False, stream=None):
    """kv_cache_append_rope into caches of 4 bits (Cache4, or pairs of their tensors; see kv_cache4).

    Without weights and cos_sin the rows are written as they are.
    """
    pages, page, heads, half = k_cache[0].shape
    cache = (pages, page, heads, 2 * half)
    d, rows, dt, dev = _append_args(K, V, slots, Q, Q_out, cos_sin, positions, q_weight, k_weight, eps, interleaved, 2 * half, heads)
    _call(dev, stream, "kv_cache4_append_rope", _entries().kv_cache4_append_rope, d, *rows, _cache4(k_cache, "k_cache", cache, dt, dev),
          _cache4(v_cache, "v_cache", cache, dt, dev), pages, page)


def kv_cache4_read(k_cache, v_cache, slots, K, V, stream=None):
    """Rows of caches of 4 bits as 16-bit values: K, V (N, H, D) from cache rows slots (N,); returns K, V."""
    pages, page, heads, half = k_cache[0].shape
    code, dev, dt, N = _dtype_code(K, "K"), K.get_device(), K.dtype, slots.numel()
    if dev < 0:
        raise ValueError("K must be a CUDA tensor")
    cache, rows = (pages, page, heads, 2 * half), (N, heads, 2 * half)
    _call(dev, stream, "kv_cache4_read", _entries().kv_cache4_read, _cache4(k_cache, "k_cache", cache, dt, dev),
          _cache4(v_cache, "v_cache", cache, dt, dev), _vector(slots, "slots", N, torch.int32, dev), _rows(K, "K", rows, dt, dev),
          _rows(V, "V", rows, dt, dev), N, heads, 2 * half, pages, page, code)
    return K, V


def tree_attention4_fwd(Q, k_cache, v_cache, block_tables, kv_lens, q_starts, parents, O, max_nodes: int,
                        softmax_scale: float = 0.0, softcap: float = 0.0, workspace=None, stream=None):
    """tree_attention_fwd over caches of 4 bits (Cache4, or pairs of their tensors); returns O.

    Q, O (N, Hq, D) of the params' type; the other arguments as there, without a distance bias.  ``workspace``: as for
    masked_attention_fwd, tree_attention4_workspace bytes (0 for little work).
    """
    code, dev, dt, i32 = _dtype_code(Q, "Q"), Q.get_device(), Q.dtype, torch.int32
    if Q.dim() != 3 or dev < 0:
        raise ValueError("Q must be a 3-D CUDA tensor (tokens, heads, head_dim)")
    N, Hq, D = Q.shape
    pages, page, heads, half = k_cache[0].shape
    cache = (pages, page, heads, D)
    if 2 * half != D:
        raise ValueError("k_cache's codes must be (pages, page_size, heads, %d), got %s" % (D // 2, tuple(k_cache[0].shape)))
    if O.shape != Q.shape or O.dtype is not dt or O.get_device() != dev:
        raise ValueError("O must be like Q")
    (qr, qh, qd), (orow, oh, od) = Q.stride(), O.stride()
    if qd != 1 or od != 1:
        raise ValueError("Q and O: the last dimension must be contiguous")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be (requests, width)")
    B, W = block_tables.shape
    d = _pack_tree(B, N, Hq, heads, D, pages, page, W, max_nodes, qr, qh, orow, oh, code, softmax_scale, softcap, 0)
    L = _entries()
    _call_scratch(dev, stream, "tree_attention4_fwd", L.tree_attention4_fwd, L.tree_attention4_workspace, workspace, d, Q.data_ptr() or None,
          _cache4(k_cache, "k_cache", cache, dt, dev), _cache4(v_cache, "v_cache", cache, dt, dev),
          _vector(block_tables, "block_tables", B * W, i32, dev), _vector(kv_lens, "kv_lens", B, i32, dev),
          _vector(q_starts, "q_starts", B + 1, i32, dev), _vector(parents, "parents", N, i32, dev), O.data_ptr() or None)
    return O


def tree_attention4_workspace(B: int, N: int, Hq: int, Hkv: int, D: int, pages: int, page_size: int, W: int, max_nodes: int) -> int:
    """Bytes of workspace a tree_attention4_fwd call of these sizes needs; 0 for little work."""
    n = lib().tree_attention4_workspace(_TreeDesc(B, N, Hq, Hkv, D, pages, page_size, W, max_nodes))
    if n < 0:
        raise GsrError(Status.ERR_INVALID_ARG, "tree_attention4_workspace")
    return n


def _probs(t, name, N, V, index):
    """The address and row stride of (N, V) float32 probabilities."""
    if t is None:
        return None, 0
    if t.dtype is not torch.float32 or t.get_device() != index or t.shape != (N, V) or (t.stride(1) != 1 and V > 1):
        raise ValueError("%s must be float32 (%d, %d) on cuda:%d with contiguous rows, got %s %s on %s"
                         % (name, N, V, index, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr() or None, t.stride(0)


def verify_drafts(target_probs, draft_tokens, q_starts, parents, u_accept, u_sample, path, counts, next_tokens,
                  draft_probs=None, stream=None):
    """Which drafted tokens the target's probabilities keep, and the token that follows; returns path, counts, next_tokens.

    Node 0 of a request is its last decided token, nodes below it are drafts (parents as in
    tree_attention_fwd; None: chains).  target_probs (N, V) float32: the target's distribution after each
    node; draft_probs: the one each node's token was drawn from (None: tokens were not drawn).  draft_tokens (N,)
    int32; u_accept (N,), u_sample (B,) float32 in [0, 1).  Writes path (B, max_nodes) int32, the kept drafts' nodes
    and then -1; counts (B,) and next_tokens (B,).  Kept and drawn tokens are distributed as the target's.
    The kept nodes' cache rows are the caller's to move together before the next step (a Cache4's codes and params).
    """
    dev, i32, f32 = target_probs.get_device(), torch.int32, torch.float32
    if dev < 0 or target_probs.dim() != 2:
        raise ValueError("target_probs must be a 2-D CUDA tensor (nodes, vocabulary)")
    N, V = target_probs.shape
    B = u_sample.numel()
    if path.dim() != 2 or path.shape[0] != B:
        raise ValueError("path must be (%d, max_nodes), got %s" % (B, tuple(path.shape)))
    (tp, ts), (dp, dr) = _probs(target_probs, "target_probs", N, V, dev), _probs(draft_probs, "draft_probs", N, V, dev)
    T = path.shape[1]
    _call(dev, stream, "verify_drafts", _entries().verify_drafts, _pack_verify(B, N, V, T, ts, dr), tp, dp,
          _vector(draft_tokens, "draft_tokens", N, i32, dev), _vector(q_starts, "q_starts", B + 1, i32, dev),
          _vector(parents, "parents", N, i32, dev), _vector(u_accept, "u_accept", N, f32, dev),
          _vector(u_sample, "u_sample", B, f32, dev), _vector(path, "path", B * T, i32, dev), _vector(counts, "counts", B, i32, dev),
          _vector(next_tokens, "next_tokens", B, i32, dev))
    return path, counts, next_tokens
