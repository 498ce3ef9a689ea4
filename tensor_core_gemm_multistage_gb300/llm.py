"""Attention of language models over libgsr: masked attention and its gradient, a paged key/value
cache's bookkeeping, and attention of drafted tokens over it.  Argument checks and marshalling
only; include/gsr.h has the full contract of each entry point."""
from __future__ import annotations

import ctypes

import torch

from .binding import GsrError, Status, lib

TREE_MAX_NODES = 64


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_int64), ("stride_head", ctypes.c_int64),
                ("stride_row", ctypes.c_int64)]


class _AttentionDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("heads_q", ctypes.c_int64), ("heads_kv", ctypes.c_int64),
                ("seq_q", ctypes.c_int64), ("seq_kv", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("causal", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p), ("doc_bounds", ctypes.c_void_p),
                ("num_docs", ctypes.c_int64), ("prefix_lens", ctypes.c_void_p)]


class _TreeDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("total_q", ctypes.c_int64), ("heads_q", ctypes.c_int64),
                ("heads_kv", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("table_width", ctypes.c_int64), ("max_nodes", ctypes.c_int64),
                ("q_stride_row", ctypes.c_int64), ("q_stride_head", ctypes.c_int64),
                ("o_stride_row", ctypes.c_int64), ("o_stride_head", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("softcap", ctypes.c_float), ("alibi_slopes", ctypes.c_void_p)]


def _declare(L) -> None:
    """Argument types of the entry points this module calls."""
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    ts, ds, tr = ctypes.POINTER(_Tensor), ctypes.POINTER(_AttentionDesc), ctypes.POINTER(_TreeDesc)
    L.masked_attention_fwd.restype = i32
    L.masked_attention_fwd.argtypes = [ds, ts, ts, ts, ts, vp, vp, i64, vp]
    L.masked_attention_fwd_workspace.restype = i64
    L.masked_attention_fwd_workspace.argtypes = [ds]
    L.masked_attention_bwd_workspace.restype = i64
    L.masked_attention_bwd_workspace.argtypes = [ds]
    L.masked_attention_bwd.restype = i32
    L.masked_attention_bwd.argtypes = [ds] + [ts] * 5 + [vp] + [ts] * 3 + [vp, i64, vp]
    L.tree_attention_workspace.restype = i64
    L.tree_attention_workspace.argtypes = [tr]
    L.tree_attention_fwd.restype = i32
    L.tree_attention_fwd.argtypes = [tr, vp, ts, ts] + [vp] * 6 + [i64, vp]
    L.kv_block_tables.restype = i32
    L.kv_block_tables.argtypes = [vp] * 11 + [i64] * 5 + [vp]
    L.kv_cache_append.restype = i32
    L.kv_cache_append.argtypes = [ts, ts, vp, ts, ts] + [i64] * 5 + [vp]


def _handle(stream, index):
    """The CUDA handle of `stream` (None: the current stream of the device), or None for the default
    stream.  The raw query is the one behind torch.cuda.current_stream, without the Stream object."""
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return (raw(index) if raw else torch.cuda.current_stream(index).cuda_stream) or None
    return (stream if isinstance(stream, int) else stream.cuda_stream) or None


# behind torch.cuda.current_device, without its look whether CUDA is there (a CUDA tensor is)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(index, stream, name, function, *args):
    """function(*args, stream handle) with the device current; raises GsrError unless it returns GSR_OK."""
    if _current_device() == index:
        s = function(*args, _handle(stream, index))
    else:
        with torch.cuda.device(index):
            s = function(*args, _handle(stream, index))
    if s != 0:
        raise GsrError(s, name)


def _dtype_code(t, name):
    if t.dtype is torch.float16:
        return 0
    if t.dtype is torch.bfloat16:
        return 1
    raise TypeError("%s must be float16 or bfloat16, got %s" % (name, t.dtype))


def _operand(t, name, shape, dtype, index):
    """The C view of a 4-D operand (batch, head, row, D) of the given shape."""
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be %s on cuda:%d, got %s on %s" % (name, dtype, index, t.dtype, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    sb, sh, sr, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return _Tensor(t.data_ptr() or None, sb, sh, sr)


def _vector(t, name, count, dtype, index):
    """The address of a contiguous device array of `count` values, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index or t.numel() != count or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of %d values on cuda:%d, got %s %s on %s"
                         % (name, dtype, count, index, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr() or None


def _scratch(workspace, nbytes, index, stream):
    """A tensor to keep until the call returns, its address and its size: the caller's workspace; None
    (the library's own for the stream); or, where the stream is being captured, a new one from the
    graph's memory."""
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on cuda:%d" % index)
        return workspace, workspace.data_ptr() or None, workspace.numel() * workspace.element_size()
    handle = _handle(stream, index)
    if handle is None:                                  # the legacy default stream cannot be captured
        return None, None, 0
    if torch.cuda.current_device() == index and (stream is None or handle == _handle(None, index)):
        if not torch.cuda.is_current_stream_capturing():
            return None, None, 0
        return _workspace(nbytes, index)
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=torch.device("cuda", index))):
        return _workspace(nbytes, index) if torch.cuda.is_current_stream_capturing() else (None, None, 0)


def _workspace(nbytes, index):
    n = max(nbytes(), 16)
    ws = torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", index))
    return ws, ws.data_ptr(), n


def _attention_desc(Q, K, softmax_scale, causal, softcap, alibi_slopes, doc_bounds, prefix_lens):
    """The C description, Q's and K's shapes, and the device."""
    code, index = _dtype_code(Q, "Q"), Q.get_device()
    if index < 0:
        raise ValueError("Q must be a CUDA tensor")
    qs, ks = Q.shape, K.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("Q and K must be 4-D (batch, heads, seq, head_dim)")
    B, Hq, Sq, D = qs
    docs = 0
    if doc_bounds is not None:
        if doc_bounds.dim() != 2 or doc_bounds.shape[0] != B or doc_bounds.shape[1] < 2:
            raise ValueError("doc_bounds must be (batch, documents + 1), got %s" % (tuple(doc_bounds.shape),))
        docs = doc_bounds.shape[1] - 1
    if prefix_lens is not None and prefix_lens.shape != (B, docs or 1) and (docs > 1 or prefix_lens.shape != (B,)):
        raise ValueError("prefix_lens must be (batch, %d), got %s" % (docs or 1, tuple(prefix_lens.shape)))
    desc = _AttentionDesc(B, Hq, ks[1], Sq, ks[2], D, code, 1 if causal else 0, softmax_scale, softcap,
                          _vector(alibi_slopes, "alibi_slopes", Hq, torch.float32, index),
                          _vector(doc_bounds, "doc_bounds", B * (docs + 1), torch.int32, index), docs,
                          _vector(prefix_lens, "prefix_lens", B * (docs or 1), torch.int32, index))
    return desc, qs, (B, ks[1], ks[2], D), index


def _lse(lse, qs, index):
    if lse is not None and lse.shape != qs[:3]:
        raise ValueError("lse must have shape %s, got %s" % (tuple(qs[:3]), tuple(lse.shape)))
    return _vector(lse, "lse", qs[0] * qs[1] * qs[2], torch.float32, index)


def masked_attention_fwd(Q, K, V, O, lse=None, softmax_scale: float = 0.0, causal: bool = False,
                         softcap: float = 0.0, alibi_slopes=None, doc_bounds=None, prefix_lens=None, workspace=None,
                         stream=None):
    """O = softmax(score) V over the keys each query sees; returns O.

    Q, O (B, Hq, Sq, D), K and V (B, Hkv, Skv, D): float16 or bfloat16 CUDA tensors, D 64 or 128 and
    contiguous, the other strides free (multiples of 8); Hq a multiple of Hkv.  ``lse``: optional
    float32 (B, Hq, Sq).  ``softcap`` c replaces the scaled product x by c tanh(x / c);
    ``alibi_slopes`` (Hq,) float32 subtracts slope * distance; ``doc_bounds`` (B, n + 1) int32 keeps
    queries inside their document (positions outside all documents are padding); ``prefix_lens``
    (B,) or (B, n) int32, with ``causal``, lets every query see that many leading keys.

    ``workspace``: optional device buffer of masked_attention_fwd_workspace(...) bytes (few queries, many
    keys); without one the library keeps one for the stream, and a call inside torch.cuda.graph takes
    one from the graph's memory.
    """
    d, qs, ks, dev = _attention_desc(Q, K, softmax_scale, causal, softcap, alibi_slopes, doc_bounds, prefix_lens)
    dt, L = Q.dtype, lib()
    ws, scratch, size = _scratch(workspace, lambda: L.masked_attention_fwd_workspace(d), dev, stream)
    _call(dev, stream, "masked_attention_fwd", L.masked_attention_fwd, d, _operand(Q, "Q", qs, dt, dev),
          _operand(K, "K", ks, dt, dev), _operand(V, "V", ks, dt, dev), _operand(O, "O", qs, dt, dev), _lse(lse, qs, dev),
          scratch, size)
    return O


def masked_attention_fwd_workspace(B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int) -> int:
    """Bytes of workspace a masked_attention_fwd call of these sizes needs, whatever its masks."""
    n = lib().masked_attention_fwd_workspace(_AttentionDesc(B, Hq, Hkv, Sq, Skv, D))
    if n < 0:
        raise GsrError(Status.ERR_INVALID_ARG, "masked_attention_fwd_workspace")
    return n


def masked_attention_bwd(dO, Q, K, V, O, lse, dQ, dK, dV, softmax_scale: float = 0.0, causal: bool = False,
                         softcap: float = 0.0, alibi_slopes=None, doc_bounds=None, prefix_lens=None, workspace=None,
                         stream=None):
    """Gradients dQ, dK, dV (returned) of masked_attention_fwd from dO, its inputs, O and lse.

    dO, O and dQ are shaped as Q, dK and dV as K; masks and scores as in the forward call.
    ``workspace``: optional device buffer of masked_attention_bwd_workspace(...) bytes, as for
    masked_attention_fwd.
    """
    d, qs, ks, dev = _attention_desc(Q, K, softmax_scale, causal, softcap, alibi_slopes, doc_bounds, prefix_lens)
    dt, L = Q.dtype, lib()
    ws, scratch, size = _scratch(workspace, lambda: L.masked_attention_bwd_workspace(d), dev, stream)
    _call(dev, stream, "masked_attention_bwd", L.masked_attention_bwd, d, _operand(dO, "dO", qs, dt, dev),
          _operand(Q, "Q", qs, dt, dev), _operand(K, "K", ks, dt, dev), _operand(V, "V", ks, dt, dev),
          _operand(O, "O", qs, dt, dev), _lse(lse, qs, dev), _operand(dQ, "dQ", qs, dt, dev),
          _operand(dK, "dK", ks, dt, dev), _operand(dV, "dV", ks, dt, dev), scratch, size)
    return dQ, dK, dV


def masked_attention_bwd_workspace(B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int) -> int:
    """Bytes of workspace a masked_attention_bwd call of these sizes needs, whatever its masks."""
    n = lib().masked_attention_bwd_workspace(_AttentionDesc(B, Hq, Hkv, Sq, Skv, D))
    if n < 0:
        raise GsrError(Status.ERR_INVALID_ARG, "masked_attention_bwd_workspace")
    return n


def _cache(t, name, shape, dtype, index):
    """The C view of a cache (pages, page_size, heads, D)."""
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError("%s must be %s on cuda:%d, got %s on %s" % (name, dtype, index, t.dtype, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    sp, sr, sh, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return _Tensor(t.data_ptr() or None, sp, sh, sr)


def tree_attention_fwd(Q, k_cache, v_cache, block_tables, kv_lens, q_starts, parents, O, max_nodes: int,
                       softmax_scale: float = 0.0, softcap: float = 0.0, alibi_slopes=None, workspace=None,
                       stream=None):
    """Attention of drafted tokens over a paged cache; returns O.

    Q, O (N, Hq, D): the drafted tokens of all requests, request b's in rows q_starts[b] to
    q_starts[b + 1]; caches (pages, page_size, Hkv, D), the drafted tokens' rows already written;
    block_tables (B, W), kv_lens (B,) with the drafted tokens, q_starts (B + 1,), parents (N,) (an
    earlier node of the request or -1; None: a chain), all int32.  A token sees what is before the
    tree, its ancestors and itself.  ``max_nodes`` bounds the nodes of one request (at most 64); 1 is
    ordinary decoding.  ``workspace``: as for masked_attention_bwd, tree_attention_workspace bytes.
    """
    code, dev, dt, i32 = _dtype_code(Q, "Q"), Q.get_device(), Q.dtype, torch.int32
    if Q.dim() != 3 or dev < 0:
        raise ValueError("Q must be a 3-D CUDA tensor (tokens, heads, head_dim)")
    N, Hq, D = Q.shape
    cache = k_cache.shape
    if len(cache) != 4 or cache[3] != D:
        raise ValueError("k_cache must be (pages, page_size, heads, %d), got %s" % (D, tuple(cache)))
    if O.shape != Q.shape or O.dtype is not dt or O.get_device() != dev:
        raise ValueError("O must be like Q")
    (qr, qh, qd), (orow, oh, od) = Q.stride(), O.stride()
    if qd != 1 or od != 1:
        raise ValueError("Q and O: the last dimension must be contiguous")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be (requests, width)")
    B, W = block_tables.shape
    d = _TreeDesc(B, N, Hq, cache[2], D, cache[0], cache[1], W, max_nodes, qr, qh, orow, oh, code, softmax_scale, softcap,
                  _vector(alibi_slopes, "alibi_slopes", Hq, torch.float32, dev))
    L = lib()
    ws, scratch, size = _scratch(workspace, lambda: L.tree_attention_workspace(d), dev, stream)
    _call(dev, stream, "tree_attention_fwd", L.tree_attention_fwd, d, Q.data_ptr() or None,
          _cache(k_cache, "k_cache", cache, dt, dev), _cache(v_cache, "v_cache", cache, dt, dev),
          _vector(block_tables, "block_tables", B * W, i32, dev), _vector(kv_lens, "kv_lens", B, i32, dev),
          _vector(q_starts, "q_starts", B + 1, i32, dev), _vector(parents, "parents", N, i32, dev),
          O.data_ptr() or None, scratch, size)
    return O


def tree_attention_workspace(B: int, N: int, Hq: int, Hkv: int, D: int, pages: int, page_size: int, W: int,
                             max_nodes: int) -> int:
    """Bytes of workspace a tree_attention_fwd call of these sizes needs."""
    n = lib().tree_attention_workspace(_TreeDesc(B, N, Hq, Hkv, D, pages, page_size, W, max_nodes))
    if n < 0:
        raise GsrError(Status.ERR_INVALID_ARG, "tree_attention_workspace")
    return n


def kv_block_tables(kv_lens, new_lens, free_blocks, free_head, block_tables, page_size: int, kv_lens_out,
                    free_head_out, q_starts, positions, slots, counts, stream=None):
    """Block tables and slot maps of one step, built on the device from the requests' lengths.

    Each request has kv_lens[b] cached tokens and gets new_lens[b] more.  Writes the entries of the
    pages it takes from free_blocks (from entry free_head[0] on) into block_tables, and kv_lens_out,
    free_head_out, q_starts (B + 1), positions and slots of the packed new tokens (-1 behind the
    last; positions as tokens are stored, which a branching tree's nodes do not have), counts = (new
    tokens, pages taken, pages missing).  All int32; nothing is read back to the host.  Returns slots.
    """
    i32, dev = torch.int32, kv_lens.get_device()
    if dev < 0:
        raise ValueError("kv_lens must be a CUDA tensor")
    B, F, N = kv_lens.numel(), free_blocks.numel(), slots.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be (%d, width), got %s" % (B, tuple(block_tables.shape)))
    W = block_tables.shape[1]
    _call(dev, stream, "kv_block_tables", lib().kv_block_tables, _vector(kv_lens, "kv_lens", B, i32, dev),
          _vector(new_lens, "new_lens", B, i32, dev), _vector(free_blocks, "free_blocks", F, i32, dev),
          _vector(free_head, "free_head", 1, i32, dev), _vector(block_tables, "block_tables", B * W, i32, dev),
          _vector(kv_lens_out, "kv_lens_out", B, i32, dev), _vector(free_head_out, "free_head_out", 1, i32, dev),
          _vector(q_starts, "q_starts", B + 1, i32, dev), _vector(positions, "positions", N, i32, dev),
          _vector(slots, "slots", N, i32, dev), _vector(counts, "counts", 3, i32, dev), B, W, page_size, F, N)
    return slots


def kv_cache_append(K, V, slots, k_cache, v_cache, stream=None):
    """Writes the rows of K and V (N, H, D) to the cache rows slots (N,) int32 names (page *
    page_size + row; negative: skipped).  Caches (pages, page_size, H, D); any 16-bit type."""
    dev, dt, cache = k_cache.get_device(), k_cache.dtype, k_cache.shape
    if dev < 0 or dt not in (torch.float16, torch.bfloat16) or len(cache) != 4:
        raise ValueError("k_cache must be a 4-D float16 or bfloat16 CUDA tensor (pages, page_size, heads, head_dim)")
    rows = K.shape
    if len(rows) != 3 or rows[1:] != cache[2:] or V.shape != rows:
        raise ValueError("K and V must be (tokens, %d, %d), got %s and %s"
                         % (cache[2], cache[3], tuple(rows), tuple(V.shape)))
    views = []
    for t, name in ((K, "K"), (V, "V")):
        row, head, one = t.stride()
        if t.dtype is not dt or t.get_device() != dev or (one != 1 and rows[2] > 1):
            raise ValueError("%s must be %s on cuda:%d with a contiguous last dimension" % (name, dt, dev))
        views.append(_Tensor(t.data_ptr() or None, 0, head, row))
    _call(dev, stream, "kv_cache_append", lib().kv_cache_append, views[0], views[1],
          _vector(slots, "slots", rows[0], torch.int32, dev), _cache(k_cache, "k_cache", cache, dt, dev),
          _cache(v_cache, "v_cache", cache, dt, dev), rows[0], rows[1], rows[2], cache[0], cache[1])
