"""Oracle of the paged key/value cache operators in fp64 (numpy), written from
their formulas: rotary positions, the append to pages, and causal attention of a
chunk of new tokens over the pages, one query row at a time."""
from __future__ import annotations

import numpy as np

PAGE = 64


def rotate(x, pos, inv_freq, rot, offset=0, neighbours=False, axis=None, inverse=False):
    """x [tokens][heads][channels] with pair i turned by pos[axis[i]] * inv_freq[i] radians."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    half = rot // 2
    axis = [0] * half if axis is None else axis
    for i in range(half):
        angle = pos[axis[i]].astype(np.float64) * np.float64(inv_freq[i])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        if inverse:
            s = -s
        ca, cb = (offset + 2 * i, offset + 2 * i + 1) if neighbours else (offset + i, offset + i + half)
        a, b = x[..., ca], x[..., cb]
        y[..., ca], y[..., cb] = a * c - b * s, b * c + a * s
    return y


def rows_of(pool, table, b, n, head):
    """Rows 0 .. n - 1 of sequence b, one kv head, in token order."""
    j = np.arange(n)
    return pool[table[b, j // PAGE], head, j % PAGE].astype(np.float64)


def append(pool, table, b, start, rows):
    """rows [m][kv_heads][channels] written behind `start` of sequence b (in place)."""
    for i, r in enumerate(rows):
        pool[table[b, (start + i) // PAGE], :, (start + i) % PAGE] = r


def attention(q, k, v, n, scale, window=0):
    """One sequence and one kv head: q [m][g][channels] stand at positions n - m .. n - 1 over k, v [n][channels].
    Returns out, lse and sum_j p_j |v_j| (the scale of the rounding errors)."""
    m, g, d = q.shape
    out, lse, mag = np.zeros((m, g, v.shape[1])), np.full((m, g), -np.inf), np.zeros((m, g, v.shape[1]))
    for i in range(m):
        p = n - m + i
        lo = max(0, p - window + 1) if window > 0 else 0
        if p < 0:
            continue
        s = scale * (q[i].astype(np.float64) @ k[lo:p + 1].T)
        top = s.max(1, keepdims=True)
        e = np.exp(s - top)
        total = e.sum(1, keepdims=True)
        out[i] = e / total @ v[lo:p + 1]
        mag[i] = e / total @ np.abs(v[lo:p + 1])
        lse[i] = (top + np.log(total))[:, 0]
    return out, lse, mag
