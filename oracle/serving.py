"""CPU oracle for head norms with rotation and their gradient, the cache of 4 bits, and the verification of
drafted tokens: numpy, fp64, the plain way.

TEST INFRASTRUCTURE ONLY (same rules as the other oracles of this package).

Definitions, written here from the formulas and sharing nothing with the library:
  * y = rot(n w), n = x / sqrt(mean(x^2) + eps): pair (a, b) of the first R columns turns to (a c - b s, b c + a s);
  * dw = sum of dy n over rows, dx = r (dy w - n mean(dy w n)) with dy the gradient turned back, r = n / x;
  * a value of 4 bits is scale x code + minimum, both for 64 values;
  * a draft is kept where u T q(x) < r(x); a refusal leaves max(r - T q, 0).
Beside results stand sums of the absolute values of their terms, from which the tests derive tolerances.
"""
from __future__ import annotations

import numpy as np

from .llm import f64


def angles(table, positions, R):
    """cos and sin (..., R / 2) of positions; rows of no position (negative) hold 0, behind the table NaN."""
    pos = np.asarray(positions, dtype=np.int64)
    rows = f64(table)[np.clip(pos, 0, len(table) - 1)]
    rows = np.where((pos >= len(table))[..., None], np.nan, rows)
    return rows[..., :R // 2], rows[..., R // 2:]


def _pairs(y, R, interleaved):
    return (y[..., 0:R:2], y[..., 1:R:2]) if interleaved else (y[..., :R // 2], y[..., R // 2:R])


def _join(c, d, rest, interleaved):
    turned = np.stack([c, d], -1).reshape(*c.shape[:-1], -1) if interleaved else np.concatenate([c, d], -1)
    return np.concatenate([turned, rest], -1)


def turn(y, cos, sin, R, interleaved=False, back=False):
    """Rotated rows and the sums of |terms|."""
    a, b = _pairs(y, R, interleaved)
    s = -sin if back else sin
    out = _join(a * cos - b * s, b * cos + a * s, y[..., R:], interleaved)
    mag = _join(np.abs(a * cos) + np.abs(b * s), np.abs(b * cos) + np.abs(a * s), np.abs(y[..., R:]), interleaved)
    return out, mag


def norm_rope(x, w=None, cos=None, sin=None, R=0, eps=1e-6, interleaved=False, padding=None):
    """x (..., D); cos, sin broadcast to (..., R / 2); padding (...) bool: rows that become 0."""
    y = f64(x)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * f64(w)
    y, mag = (y, np.abs(y)) if cos is None else turn(y, cos, sin, R, interleaved)
    if padding is not None:
        y, mag = np.where(padding[..., None], 0.0, y), np.where(padding[..., None], 0.0, mag)
    return y, mag


def norm_rope_bwd(do, x, w=None, cos=None, sin=None, R=0, eps=1e-6, interleaved=False, padding=None):
    """(dx, |terms|), (dw, |terms|); dw is None without w.  Everything but the last axis is summed in dw."""
    dy = f64(do)
    dy, mag = (dy, np.abs(dy)) if cos is None else turn(dy, cos, sin, R, interleaved, back=True)
    if padding is not None:
        gone = np.broadcast_to(padding[..., None], dy.shape)
        dy, mag = np.where(gone, 0.0, dy), np.where(gone, 0.0, mag)
    if w is None:
        return (dy, mag), None
    x = f64(x)
    if padding is not None:
        x = np.where(gone, 0.0, x)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, dn, dn_mag = x * r, dy * f64(w), mag * np.abs(f64(w))
    dx = r * (dn - n * (dn * n).mean(-1, keepdims=True))
    dx_mag = r * (dn_mag + np.abs(n) * (dn_mag * np.abs(n)).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return (dx, dx_mag), ((dy * n).sum(axes), (mag * np.abs(n)).sum(axes))


def values4(codes, params):
    """The values (..., D) that codes (..., D / 2) and params (..., D / 64, 2) stand for, and s |c - 8| + |m + 8 s|."""
    codes, params = np.asarray(codes, dtype=np.int64), f64(params)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1, 64)
    s, m = params[..., :1], params[..., 1:]
    flat = lambda a: a.reshape(*codes.shape[:-1], -1)
    return flat(s * c + m), flat(s * np.abs(c - 8) + np.abs(m + 8 * s))


def _sane(row):
    return np.clip(np.nan_to_num(f64(row), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)


def verify(target, draft, tokens, starts, parents, u_accept, u_sample, max_nodes):
    """Request by request: lists of kept nodes, and next tokens (-1: none)."""
    target, tokens = f64(target), [int(x) for x in tokens]
    paths, nexts = [], []
    for b in range(len(starts) - 1):
        q0, T = int(starts[b]), min(int(starts[b + 1]) - int(starts[b]), max_nodes)
        path, cur, at, T_left = [], 0, 1, 1.0
        if T <= 0:
            paths.append([])
            nexts.append(-1)
            continue
        r = _sane(target[q0])
        while at < T:
            c, at = at, at + 1
            up = c - 1 if parents is None else int(parents[q0 + c])
            if up != cur or up < 0 or up >= c:
                continue
            x, u = tokens[q0 + c], float(u_accept[q0 + c])
            known = 0 <= x < target.shape[1]
            q = None if draft is None else _sane(draft[q0 + c])
            if known and u * T_left * (1.0 if q is None else q[x]) < r[x]:
                path.append(c)
                cur, r, T_left = c, _sane(target[q0 + c]), 1.0
            elif q is None:
                if known:
                    T_left -= r[x]
                    r = r.copy()
                    r[x] = 0.0
            else:
                r = np.maximum(r - T_left * q, 0.0)
                T_left = r.sum()
        if not r.sum() > 0:
            r = _sane(target[q0 + cur])
        sums = np.cumsum(r)
        paths.append(path)
        nexts.append(int(np.searchsorted(sums, float(u_sample[b]) * sums[-1], side="right")) if sums[-1] > 0 else -1)
    return paths, nexts
