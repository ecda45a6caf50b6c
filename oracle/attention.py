"""The attention block between the QKV and the output projection, in fp64: head norms with
rotation, their gradients, the append to a paged cache, drafted trees and attention over the
cache.  Written from the definitions; shares no code with the HIP path.

``cos_sin`` is the rotation table [positions, rot] (rot / 2 cosines, then the sines).  Heads
are [T, heads, D]; a paged cache is [pages, kv heads, page size, D].  ``positions`` are [T], or
with ``axes`` (an axis for each pair) [axes, T].
"""

from __future__ import annotations

import numpy as np

__all__ = ["rotate", "norm_rope", "norm_rope_backward", "append", "tree_mask", "tree_attention"]


def _pairs(rot: int, interleaved: bool):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, positions, cos_sin, interleaved=False, sign=1.0, axes=None):
    """Each head's pairs turned by sign times the position's angles."""
    y = np.array(x, np.float64)
    if cos_sin is None:
        return y
    cos_sin = np.asarray(cos_sin, np.float64)
    rot = cos_sin.shape[1]
    a, b = _pairs(rot, interleaved)
    if axes is None:
        angles = cos_sin[positions]
    else:  # pair i by its own axis
        row, pair = np.asarray(positions)[list(axes)].T, np.arange(rot // 2)
        angles = np.concatenate([cos_sin[row, pair], cos_sin[row, rot // 2 + pair]], 1)
    c, s = angles[:, None, :rot // 2], sign * angles[:, None, rot // 2:]
    ya, yb = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y


def norm_rope(x, positions, cos_sin, weight, eps, interleaved=False, axes=None):
    """Norm (weight not None) and rotation of heads [T, H, D]."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    return rotate(x, positions, cos_sin, interleaved, axes=axes)


def norm_rope_backward(x, dy, positions, cos_sin, weight, eps, interleaved=False, axes=None):
    """(dx, dweight) of :func:`norm_rope` (dweight None without a weight)."""
    g = rotate(dy, positions, cos_sin, interleaved, sign=-1.0, axes=axes)
    if weight is None:
        return g, None
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    gw = g * np.asarray(weight, np.float64)
    return r * (gw - xh * (gw * xh).mean(-1, keepdims=True)), (g * xh).sum((0, 1))


def append(cache, rows, slots):
    """Rows [T, kv heads, D] written to their slots of a copy of ``cache`` (negative: left out)."""
    out = np.array(cache, np.float64)
    page = out.shape[2]
    for t, s in enumerate(slots):
        if s >= 0:
            out[s // page, :, s % page] = rows[t]
    return out


def tree_mask(parents, q_indptr):
    """Sets of drafted tokens each token sees: itself and its ancestors, as Python integers."""
    rows = []
    for b in range(len(q_indptr) - 1):
        own = []
        for j, p in enumerate(parents[q_indptr[b]:q_indptr[b + 1]]):
            own.append((own[p] if p >= 0 else 0) | (1 << j))
        rows += own
    return rows


def tree_attention(q, k_cache, v_cache, page_table, kv_len, q_indptr, masks, scale):
    """(out [T, n_q, D], lse [T, n_q], weighted [T, n_q, D], spread [T, n_q]): the attention of
    each drafted token; ``masks`` per token a Python integer of the drafted tokens it sees, or
    None for causal order.  ``weighted`` is the softmax average of |V| and ``spread`` the largest
    sum of |q||k| scale, the scales of the rounding errors that a test allows for.  Keys that
    a token does not see do not enter, whatever they hold."""
    q = np.asarray(q, np.float64)
    T, n_q, D = q.shape
    page, n_kv = k_cache.shape[2], k_cache.shape[1]
    G = n_q // n_kv
    out, lse = np.zeros((T, n_q, D)), np.full((T, n_q), -np.inf)
    weighted, spread = np.zeros((T, n_q, D)), np.zeros((T, n_q))
    for b in range(len(kv_len)):
        kv, q0, q1 = int(kv_len[b]), int(q_indptr[b]), int(q_indptr[b + 1])
        n = q1 - q0
        if n == 0 or kv == 0:
            continue
        pages = np.asarray(page_table[b][:-(-kv // page)])
        for h in range(n_kv):
            k = k_cache[pages, h].reshape(-1, D)[:kv]
            v = v_cache[pages, h].reshape(-1, D)[:kv]
            for j in range(n):
                m = (1 << (j + 1)) - 1 if masks is None else masks[q0 + j]
                seen = np.array([True] * (kv - n) + [bool(m >> i & 1) for i in range(n)])
                if not seen.any():
                    continue
                ks, vs = k[seen], v[seen]
                for i in range(h * G, (h + 1) * G):
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = ks @ q[q0 + j, i] * scale
                        mx = s.max()
                        p = np.exp(s - mx)
                        out[q0 + j, i] = p @ vs / p.sum()
                        lse[q0 + j, i] = mx + np.log(p.sum())
                        weighted[q0 + j, i] = p @ np.abs(vs) / p.sum()
                        spread[q0 + j, i] = (np.abs(ks) @ np.abs(q[q0 + j, i])).max() * abs(scale)
    return out, lse, weighted, spread
