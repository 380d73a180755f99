"""fp64 oracle of the operators around the caches (test infrastructure): head norms with
rotary positions, the slots of appended tokens, dense attention of packed rows, and the
merge of a shared prefix with a sequence's own part. Plain numpy; shares no code with the
CUDA path. Each function also returns what its error bound needs."""
from __future__ import annotations

import numpy as np


def norm_rope(x, positions, frequencies=None, interleaved=False, factor=1.0, weight=None,
              eps=0.0, norm=False):
    """x [N, H, d] -> (y, size): the normed and rotated heads, and per element the sum of the
    magnitudes that it is a difference of."""
    x = np.asarray(x, dtype=np.float64)
    if norm:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        if weight is not None:
            x = x * np.asarray(weight, dtype=np.float64)
    y, size = x.copy(), np.abs(x)
    if frequencies is None or len(frequencies) == 0:
        return y, size
    half = len(frequencies)
    for i, f in enumerate(np.asarray(frequencies, dtype=np.float64)):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = np.asarray(positions, dtype=np.float64) * f
        c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = abs(factor) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


def row_tokens(cu, lens, N):
    """(sequence, token number) of each of N rows; (-1, -1): padding."""
    out = []
    for n in range(N):
        b = next((b for b in range(len(lens)) if cu[b] <= n < cu[b + 1]), -1)
        out.append((b, -1) if b < 0 else (b, int(lens[b]) - (int(cu[b + 1]) - n)))
    return out


def attend_rows(q, K, V, scale, visible):
    """Query rows q [n, d] of one head over the keys with visible[i, j]: (o, lse, spread, size),
    where spread [n, d] = sum_j p_j |v_j| (what relative errors of the p_j are relative to) and
    size [n] = the largest scale * sum_c |q_c k_jc| of the row (what rounding errors of its
    scores are relative to)."""
    q, K, V = (np.asarray(x, dtype=np.float64) for x in (q, K, V))
    visible = np.asarray(visible, dtype=bool)
    used = visible.any(0)             # keys that nobody sees may hold anything
    K, V, visible = K[used], V[used], visible[:, used]
    if K.shape[0] == 0:
        n = q.shape[0]
        return np.zeros(q.shape), np.full(n, -np.inf), np.zeros(q.shape), np.zeros(n)
    s = np.where(visible, q @ K.T * scale, -np.inf)
    m = s.max(1, keepdims=True)
    some = np.isfinite(m)
    p = np.exp(s - np.where(some, m, 0.0))
    l = p.sum(1, keepdims=True)
    p = p / np.where(l > 0, l, 1.0)
    lse = np.where(some, np.where(some, m, 0.0) + np.log(np.where(l > 0, l, 1.0)), -np.inf)[:, 0]
    size = np.where(visible, np.abs(q) @ np.abs(K).T * scale, 0.0).max(1)
    return p @ V, lse, p @ np.abs(V), size


def merge(o_a, lse_a, o_b, lse_b):
    """Attention over two disjoint key sets from the attention over each: (o, lse, wa, wb),
    with the weights of the two. o [..., d], lse [...]."""
    o_a, o_b = np.asarray(o_a, dtype=np.float64), np.asarray(o_b, dtype=np.float64)
    lse_a, lse_b = np.asarray(lse_a, dtype=np.float64), np.asarray(lse_b, dtype=np.float64)
    m = np.maximum(lse_a, lse_b)
    base = np.where(np.isfinite(m), m, 0.0)
    a, b = np.exp(lse_a - base), np.exp(lse_b - base)
    l = np.where(a + b > 0, a + b, 1.0)
    wa, wb = a / l, b / l
    # a part of weight 0 may hold anything
    o = (np.where(wa[..., None] > 0, o_a, 0.0) * wa[..., None]
         + np.where(wb[..., None] > 0, o_b, 0.0) * wb[..., None])
    return o, np.where(np.isfinite(m), base + np.log(l), -np.inf), wa, wb
