"""Attention of language models over libgsr: masked attention and its gradient, a paged key/value
cache's bookkeeping, and attention of drafted tokens over it.  Argument checks and marshalling
only; include/gsr.h has the full contract of each entry point."""
from __future__ import annotations

import ctypes

from .binding import GsrError, Status, _stream_handle, lib

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
    L.masked_attention_fwd.argtypes = [ds, ts, ts, ts, ts, vp, vp]
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


def _call(dev, stream, name, run):
    """run(library, stream handle) with `dev` current; raises GsrError unless it returns GSR_OK."""
    import torch
    L = lib()
    if torch.cuda.current_device() == dev.index:
        s = run(L, _stream_handle(stream, dev) or None)
    else:
        with torch.cuda.device(dev):
            s = run(L, _stream_handle(stream, dev) or None)
    if s != Status.OK:
        raise GsrError(s, name)


def _dtype_code(t, name):
    import torch
    if t.dtype == torch.float16:
        return 0
    if t.dtype == torch.bfloat16:
        return 1
    raise TypeError("%s must be float16 or bfloat16, got %s" % (name, t.dtype))


def _operand(t, name, shape, dtype, dev):
    """The C view of a 4-D operand (batch, head, row, D) of the given shape."""
    if t.dtype != dtype or t.device != dev:
        raise ValueError("%s must be %s on %s, got %s on %s" % (name, dtype, dev, t.dtype, t.device))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    sb, sh, sr, sd = t.stride()
    if sd != 1 and shape[3] > 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return _Tensor(t.data_ptr() or None, sb, sh, sr)


def _vector(t, name, shape, dtype, dev):
    """The address of a contiguous device array of the given shape, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.device != dev or not t.is_contiguous() or tuple(t.shape) not in shape:
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s, got %s %s on %s"
                         % (name, dtype, " or ".join(str(s) for s in shape), dev, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr() or None


def _scratch(workspace, nbytes, dev, stream):
    """The caller's workspace, or a new one that lives until the work queued on `stream` is done."""
    import torch
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % dev)
        return workspace
    ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
    if stream is not None:
        ws.record_stream(torch.cuda.ExternalStream(stream, device=dev) if isinstance(stream, int) else stream)
    return ws


def _attention_desc(Q, K, softmax_scale, causal, softcap, alibi_slopes, doc_bounds, prefix_lens):
    import torch
    code = _dtype_code(Q, "Q")
    if Q.dim() != 4 or K.dim() != 4:
        raise ValueError("Q and K must be 4-D (batch, heads, seq, head_dim)")
    B, Hq, Sq, D = Q.shape
    Hkv, Skv = K.shape[1], K.shape[2]
    dev = Q.device
    if dev.type != "cuda":
        raise ValueError("Q must be a CUDA tensor")
    docs = 0
    if doc_bounds is not None:
        if doc_bounds.dim() != 2 or doc_bounds.shape[1] < 2:
            raise ValueError("doc_bounds must be (batch, documents + 1), got %s" % (tuple(doc_bounds.shape),))
        docs = doc_bounds.shape[1] - 1
    prefix_shapes = ((B, max(docs, 1)), (B,)) if docs <= 1 else ((B, docs),)
    return _AttentionDesc(
        B, Hq, Hkv, Sq, Skv, D, code, 1 if causal else 0, softmax_scale, softcap,
        _vector(alibi_slopes, "alibi_slopes", ((Hq,),), torch.float32, dev),
        _vector(doc_bounds, "doc_bounds", ((B, docs + 1),), torch.int32, dev), docs,
        _vector(prefix_lens, "prefix_lens", prefix_shapes, torch.int32, dev)), (B, Hq, Sq, D), (B, Hkv, Skv, D)


def masked_attention_fwd(Q, K, V, O, lse=None, softmax_scale: float = 0.0, causal: bool = False,
                         softcap: float = 0.0, alibi_slopes=None, doc_bounds=None, prefix_lens=None, stream=None):
    """O = softmax(score) V over the keys each query sees; returns O.

    Q, O (B, Hq, Sq, D), K and V (B, Hkv, Skv, D): float16 or bfloat16 CUDA tensors, D 64 or 128 and
    contiguous, the other strides free (multiples of 8); Hq a multiple of Hkv.  ``lse``: optional
    float32 (B, Hq, Sq).  ``softcap`` c replaces the scaled product x by c tanh(x / c);
    ``alibi_slopes`` (Hq,) float32 subtracts slope * distance; ``doc_bounds`` (B, n + 1) int32 keeps
    queries inside their document (positions outside all documents are padding); ``prefix_lens``
    (B,) or (B, n) int32, with ``causal``, lets every query see that many leading keys.
    """
    import torch
    d, qs, ks = _attention_desc(Q, K, softmax_scale, causal, softcap, alibi_slopes, doc_bounds, prefix_lens)
    dt, dev = Q.dtype, Q.device
    args = [_operand(Q, "Q", qs, dt, dev), _operand(K, "K", ks, dt, dev), _operand(V, "V", ks, dt, dev),
            _operand(O, "O", qs, dt, dev)]
    lse_ptr = _vector(lse, "lse", (qs[:3],), torch.float32, dev)
    _call(dev, stream, "masked_attention_fwd", lambda L, st: L.masked_attention_fwd(d, *args, lse_ptr, st))
    return O


def masked_attention_bwd(dO, Q, K, V, O, lse, dQ, dK, dV, softmax_scale: float = 0.0, causal: bool = False,
                         softcap: float = 0.0, alibi_slopes=None, doc_bounds=None, prefix_lens=None, workspace=None,
                         stream=None):
    """Gradients dQ, dK, dV (returned) of masked_attention_fwd from dO, its inputs, O and lse.

    dO, O and dQ are shaped as Q, dK and dV as K; masks and scores as in the forward call.
    ``workspace``: optional device buffer of masked_attention_bwd_workspace(...) bytes; without one
    the call takes it from PyTorch's allocator.
    """
    import torch
    d, qs, ks = _attention_desc(Q, K, softmax_scale, causal, softcap, alibi_slopes, doc_bounds, prefix_lens)
    dt, dev = Q.dtype, Q.device
    dO_, Q_, O_, dQ_ = (_operand(t, n, qs, dt, dev) for t, n in ((dO, "dO"), (Q, "Q"), (O, "O"), (dQ, "dQ")))
    K_, V_, dK_, dV_ = (_operand(t, n, ks, dt, dev) for t, n in ((K, "K"), (V, "V"), (dK, "dK"), (dV, "dV")))
    lse_ptr = _vector(lse, "lse", (qs[:3],), torch.float32, dev)
    need = lib().masked_attention_bwd_workspace(d)
    ws = _scratch(workspace, need, dev, stream)
    _call(dev, stream, "masked_attention_bwd",
          lambda L, st: L.masked_attention_bwd(d, dO_, Q_, K_, V_, O_, lse_ptr, dQ_, dK_, dV_, ws.data_ptr(),
                                               ws.numel() * ws.element_size(), st))
    return dQ, dK, dV


def masked_attention_bwd_workspace(B: int, Hq: int, Hkv: int, Sq: int, Skv: int, D: int) -> int:
    """Bytes of workspace a masked_attention_bwd call of these sizes needs."""
    n = lib().masked_attention_bwd_workspace(_AttentionDesc(B, Hq, Hkv, Sq, Skv, D))
    if n < 0:
        raise GsrError(Status.ERR_INVALID_ARG, "masked_attention_bwd_workspace")
    return n


def _cache(t, name, H, D, dtype, dev):
    """The C view of a cache (pages, page_size, heads, D)."""
    if t.dtype != dtype or t.device != dev:
        raise ValueError("%s must be %s on %s, got %s on %s" % (name, dtype, dev, t.dtype, t.device))
    if t.dim() != 4 or t.shape[2] != H or t.shape[3] != D:
        raise ValueError("%s must be (pages, page_size, %d, %d), got %s" % (name, H, D, tuple(t.shape)))
    sp, sr, sh, sd = t.stride()
    if sd != 1 and D > 1:
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
    ordinary decoding.
    """
    import torch
    code, dev = _dtype_code(Q, "Q"), Q.device
    if Q.dim() != 3 or dev.type != "cuda":
        raise ValueError("Q must be a 3-D CUDA tensor (tokens, heads, head_dim)")
    N, Hq, D = Q.shape
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must be 4-D of one shape, got %s and %s"
                         % (tuple(k_cache.shape), tuple(v_cache.shape)))
    pages, page, Hkv = k_cache.shape[:3]
    if O.shape != Q.shape or O.dtype != Q.dtype or O.device != dev:
        raise ValueError("O must be like Q")
    (qr, qh, qd), (orow, oh, od) = Q.stride(), O.stride()
    if qd != 1 or od != 1:
        raise ValueError("Q and O: the last dimension must be contiguous")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be (requests, width)")
    B, W = block_tables.shape
    i32 = torch.int32
    K_, V_ = _cache(k_cache, "k_cache", Hkv, D, Q.dtype, dev), _cache(v_cache, "v_cache", Hkv, D, Q.dtype, dev)
    ptrs = [_vector(block_tables, "block_tables", ((B, W),), i32, dev), _vector(kv_lens, "kv_lens", ((B,),), i32, dev),
            _vector(q_starts, "q_starts", ((B + 1,),), i32, dev), _vector(parents, "parents", ((N,),), i32, dev)]
    d = _TreeDesc(B, N, Hq, Hkv, D, pages, page, W, max_nodes, qr, qh, orow, oh, code, softmax_scale, softcap,
                  _vector(alibi_slopes, "alibi_slopes", ((Hq,),), torch.float32, dev))
    need = lib().tree_attention_workspace(d)
    ws = _scratch(workspace, need, dev, stream)
    _call(dev, stream, "tree_attention_fwd",
          lambda L, st: L.tree_attention_fwd(d, Q.data_ptr() or None, K_, V_, *ptrs, O.data_ptr() or None,
                                             ws.data_ptr(), ws.numel() * ws.element_size(), st))
    return O


def kv_block_tables(kv_lens, new_lens, free_blocks, free_head, block_tables, page_size: int, kv_lens_out,
                    free_head_out, q_starts, positions, slots, counts, stream=None):
    """Block tables and slot maps of one step, built on the device from the requests' lengths.

    Each request has kv_lens[b] cached tokens and gets new_lens[b] more.  Writes the entries of the
    pages it takes from free_blocks (from entry free_head[0] on) into block_tables, and kv_lens_out,
    free_head_out, q_starts (B + 1), positions and slots of the packed new tokens (-1 behind the
    last), counts = (new tokens, pages taken, pages missing).  All int32; nothing is read back to the
    host.  Returns slots.
    """
    import torch
    i32, dev = torch.int32, kv_lens.device
    if dev.type != "cuda":
        raise ValueError("kv_lens must be a CUDA tensor")
    B = kv_lens.shape[0]
    W, F, N = block_tables.shape[-1], free_blocks.shape[0], slots.shape[0]
    ptrs = [_vector(t, n, (s,), i32, dev) for t, n, s in (
        (kv_lens, "kv_lens", (B,)), (new_lens, "new_lens", (B,)), (free_blocks, "free_blocks", (F,)),
        (free_head, "free_head", (1,)), (block_tables, "block_tables", (B, W)), (kv_lens_out, "kv_lens_out", (B,)),
        (free_head_out, "free_head_out", (1,)), (q_starts, "q_starts", (B + 1,)), (positions, "positions", (N,)),
        (slots, "slots", (N,)), (counts, "counts", (3,)))]
    _call(dev, stream, "kv_block_tables", lambda L, st: L.kv_block_tables(*ptrs, B, W, page_size, F, N, st))
    return slots


def kv_cache_append(K, V, slots, k_cache, v_cache, stream=None):
    """Writes the rows of K and V (N, H, D) to the cache rows slots (N,) int32 names (page *
    page_size + row; negative: skipped).  Caches (pages, page_size, H, D); any 16-bit type."""
    import torch
    dev, dt = k_cache.device, k_cache.dtype
    if dev.type != "cuda" or dt not in (torch.float16, torch.bfloat16):
        raise ValueError("k_cache must be a float16 or bfloat16 CUDA tensor")
    if K.dim() != 3 or K.shape != V.shape:
        raise ValueError("K and V must be (tokens, heads, head_dim), got %s and %s" % (tuple(K.shape), tuple(V.shape)))
    N, H, D = K.shape
    views = []
    for t, name in ((K, "K"), (V, "V")):
        if t.dtype != dt or t.device != dev or (t.stride(2) != 1 and D > 1):
            raise ValueError("%s must be %s on %s with a contiguous last dimension" % (name, dt, dev))
        views.append(_Tensor(t.data_ptr() or None, 0, t.stride(1), t.stride(0)))
    kc, vc = _cache(k_cache, "k_cache", H, D, dt, dev), _cache(v_cache, "v_cache", H, D, dt, dev)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache differ in shape")
    at = _vector(slots, "slots", ((N,),), torch.int32, dev)
    _call(dev, stream, "kv_cache_append",
          lambda L, st: L.kv_cache_append(*views, at, kc, vc, N, H, D, k_cache.shape[0], k_cache.shape[1], st))
