"""CPU oracle for masked attention and its gradient, attention of drafted tokens over a paged
cache, block tables and cache writes: numpy, fp64, the plain way.

TEST INFRASTRUCTURE ONLY (same rules as the other oracles of this package).

Definitions, written here from the formulas and sharing nothing with the library:
  * query i of a row stands at p = i + (Skv - Sq); it sees the keys of its document (all keys without
    documents), under a causal mask only those with j <= p or inside the prefix of its document;
  * score = scale q.k, capped as cap tanh(score / cap), minus slope |p - j|;
  * a query that sees nothing has output 0 and log-sum-exp -inf;
  * dV = P^T dO, dS = P (dO V^T - delta) (1 - tanh^2), dQ = scale dS K, dK = scale dS^T Q, with
    P = exp(score - lse) and delta = rowsum(dO O) from the given lse and O.
Beside each result stands the sum of the absolute values of its terms, from which the tests derive
their tolerances.
"""
from __future__ import annotations

import numpy as np


def f64(x):
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def visible(B, Sq, Skv, causal=False, doc_bounds=None, prefix_lens=None):
    """(B, Sq, Skv) bool."""
    out = np.zeros((B, Sq, Skv), dtype=bool)
    for b in range(B):
        if doc_bounds is None:
            spans = [(0, Skv, range(Sq))]
        else:
            spans = [(int(s), int(e), range(int(s), int(e))) for s, e in zip(doc_bounds[b][:-1], doc_bounds[b][1:])]
        for d, (s, e, rows) in enumerate(spans):
            for i in rows:
                for j in range(s, e):
                    ok = not causal or j <= i + Skv - Sq
                    if prefix_lens is not None and j < s + int(np.ravel(prefix_lens[b])[d]):
                        ok = True
                    out[b, i, j] = ok
    return out


def _scores(Q, K, scale, cap, slopes):
    B, Hq, Sq, D = Q.shape
    Skv, g = K.shape[2], Hq // K.shape[1]
    if not scale:
        scale = 1.0 / np.sqrt(D)
    Kg = np.repeat(K, g, axis=1)
    x = np.einsum("bhqd,bhkd->bhqk", Q, Kg) * scale
    t = np.zeros_like(x)
    if cap:
        t = np.tanh(x / cap)
        x = cap * t
    if slopes is not None:
        dist = np.abs(np.arange(Sq)[:, None] + (Skv - Sq) - np.arange(Skv)[None, :])
        x = x - f64(slopes)[None, :, None, None] * dist
    return x, t, Kg, scale


def masked_attention(Q, K, V, see, scale=0.0, cap=0.0, slopes=None):
    """(O, lse, sum of |terms| of O) in fp64; inputs may hold NaN where nothing sees them."""
    Q, K, V = f64(Q), f64(K), f64(V)
    with np.errstate(invalid="ignore", over="ignore"):
        x, _, _, _ = _scores(Q, K, scale, cap, slopes)
    x = np.where(see[:, None], x, -np.inf)
    m = x.max(axis=-1, keepdims=True) if x.shape[-1] else np.full(x.shape[:-1] + (1,), -np.inf)
    m = np.where(m == -np.inf, 0.0, m)
    p = np.exp(x - m)
    l = p.sum(-1, keepdims=True)
    p = p / np.where(l == 0, 1.0, l)
    Vg = np.repeat(V, Q.shape[1] // K.shape[1], axis=1)
    Vs = np.where(np.isfinite(Vg), Vg, 0.0)          # a NaN that is seen is not tested this way
    with np.errstate(divide="ignore"):
        lse = m[..., 0] + np.log(l[..., 0])
    return np.einsum("bhqk,bhkd->bhqd", p, Vs), lse, np.einsum("bhqk,bhkd->bhqd", p, np.abs(Vs))


def masked_attention_bwd(dO, Q, K, V, O, lse, see, scale=0.0, cap=0.0, slopes=None):
    """((dQ, dK, dV), three sums of |terms| of each: over P or |dS| (the rounded factor), with dS's own
    two terms apart, and with 1 in place of the rounded factor)."""
    dO, Q, K, V, O, lse = (f64(t) for t in (dO, Q, K, V, O, lse))
    B, Hq, Sq, D = Q.shape
    Hkv, Skv = K.shape[1], K.shape[2]
    g = Hq // Hkv
    clean = lambda t: np.where(np.isfinite(t), t, 0.0)
    empty = ~see.any(-1)                                                  # (B, Sq)
    dO, Q, K, V, O = clean(dO), clean(Q), clean(K), clean(V), clean(O)
    dO = np.where(empty[:, None, :, None], 0.0, dO)
    x, t, Kg, scale = _scores(Q, K, scale, cap, slopes)
    Vg = np.repeat(V, g, axis=1)
    with np.errstate(invalid="ignore"):
        P = np.where(see[:, None], np.exp(np.where(see[:, None], x - np.where(np.isfinite(lse), lse, 0.0)[..., None], -np.inf)), 0.0)
    dP = np.einsum("bhqd,bhkd->bhqk", dO, Vg)
    aP = np.einsum("bhqd,bhkd->bhqk", np.abs(dO), np.abs(Vg))
    delta, adelta = (dO * O).sum(-1)[..., None], np.abs(dO * O).sum(-1)[..., None]
    dS = P * (dP - delta) * (1 - t * t)
    aS = P * (aP + adelta)
    fold = lambda a: a.reshape(B, Hkv, g, Skv, D).sum(2)
    dQ = scale * np.einsum("bhqk,bhkd->bhqd", dS, Kg)
    dK = scale * fold(np.einsum("bhqk,bhqd->bhkd", dS, Q))
    dV = fold(np.einsum("bhqk,bhqd->bhkd", P, dO))
    terms = (abs(scale) * np.einsum("bhqk,bhkd->bhqd", np.abs(dS), np.abs(Kg)),
             abs(scale) * fold(np.einsum("bhqk,bhqd->bhkd", np.abs(dS), np.abs(Q))),
             fold(np.einsum("bhqk,bhqd->bhkd", P, np.abs(dO))))
    wide = (abs(scale) * np.einsum("bhqk,bhkd->bhqd", aS, np.abs(Kg)),
            abs(scale) * fold(np.einsum("bhqk,bhqd->bhkd", aS, np.abs(Q))), terms[2])
    seen = np.repeat(see[:, None], Hq, axis=1).astype(np.float64)
    plain = (abs(scale) * np.einsum("bhqk,bhkd->bhqd", seen, np.abs(Kg)),
             abs(scale) * fold(np.einsum("bhqk,bhqd->bhkd", seen, np.abs(Q))),
             fold(np.einsum("bhqk,bhqd->bhkd", seen, np.abs(dO))))
    return (dQ, dK, dV), terms, wide, plain


def tree_attention(Q, k_cache, v_cache, table, kv_lens, q_starts, parents, scale=0.0, cap=0.0, slopes=None,
                   max_nodes=64):
    """(O (N, Hq, D), sum of |terms|) ; rows no request computes are NaN."""
    Q = f64(Q)
    N, Hq, D = Q.shape
    pages, page, Hkv = k_cache.shape[:3]
    kc, vc = f64(k_cache), f64(v_cache)
    scale = scale or 1.0 / np.sqrt(D)
    out = np.full((N, Hq, D), np.nan)
    terms = np.full((N, Hq, D), np.nan)
    for b in range(len(kv_lens)):
        s, e = int(q_starts[b]), int(q_starts[b + 1])
        kv, T = int(kv_lens[b]), e - s
        ctx = kv - T
        for t in range(min(T, max_nodes)):
            chain, u = [t], t
            while True:
                up = u - 1 if parents is None else int(parents[s + u])
                if up < 0 or up >= u:
                    break
                chain.append(up)
                u = up
            chain.reverse()
            keys = [(j, j) for j in range(max(ctx, 0))] + [(ctx + u, ctx + d) for d, u in enumerate(chain) if ctx + u >= 0]
            pos = ctx + len(chain) - 1
            rows, at = [], []
            for j, where in keys:
                col = j // page
                if j >= kv or col >= table.shape[1] or not 0 <= int(table[b][col]) < pages:
                    continue
                rows.append((int(table[b][col]), j % page))
                at.append(where)
            if not rows:
                out[s + t], terms[s + t] = 0.0, 0.0
                continue
            pg, off = np.array(rows).T
            for h in range(Hq):
                k, v = kc[pg, off, h * Hkv // Hq], vc[pg, off, h * Hkv // Hq]
                x = k @ Q[s + t, h] * scale
                if cap:
                    x = cap * np.tanh(x / cap)
                if slopes is not None:
                    x = x - float(slopes[h]) * (pos - np.array(at, dtype=np.float64))
                p = np.exp(x - x.max())
                p /= p.sum()
                out[s + t, h], terms[s + t, h] = p @ v, p @ np.abs(v)
    return out, terms


def block_tables(kv_lens, new_lens, free_blocks, head, table, page, max_tokens):
    """Dict of the call's outputs, request by request and token by token."""
    table = np.array(table, dtype=np.int64)
    B, W = table.shape
    head = min(max(int(head), 0), len(free_blocks))
    starts, slots, positions = [0], [], []
    taken = missing = 0
    for b in range(B):
        old, new = max(int(kv_lens[b]), 0), max(int(new_lens[b]), 0)
        for pos in range(old, old + new):
            col = pos // page
            if pos % page == 0 or pos == old:
                if col >= -(-old // page):                # a page this step opens
                    if pos % page == 0:
                        if col >= W:
                            missing += 1
                        elif head < len(free_blocks):
                            table[b, col] = free_blocks[head]
                            head += 1
                            taken += 1
                        else:
                            table[b, col] = -1
                            missing += 1
            block = table[b, col] if col < W else -1
            slots.append(block * page + pos % page if block >= 0 else -1)
            positions.append(pos)
        starts.append(starts[-1] + new)
    total = len(slots)
    pad = lambda a: np.array((a + [-1] * max_tokens)[:max_tokens], dtype=np.int64)
    return {"table": table, "kv_out": np.array([max(int(a), 0) + max(int(n), 0) for a, n in zip(kv_lens, new_lens)]),
            "head_out": np.array([head]), "q_starts": np.array(starts), "positions": pad(positions),
            "slots": pad(slots), "counts": np.array([total, taken, missing])}
