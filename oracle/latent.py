"""Latent attention over a paged cache (oracle; test infrastructure only).

All heads of a token share one latent vector c [R] and one rotated key part k [64], which
is what a cached row holds, side by side.  Everything here is a restatement of the
formulas in float64, request by request and row by row:

  append    cache[slot] = (norm(c), rot(k)),  norm(x) = x w / sqrt(mean(x^2) + eps)
  gather    rows of a sequence in order
  absorbed  out[t][h] = sum_j p_j c_j,  p = softmax(scale (a . c_j + b . k_j)),  q = (a, b)
  expanded  out[t][h] = sum_j p_j v_jh, p = softmax(scale (a . k_jh + b . r_j)), q = (a, b)

The rotation is a decision of the cache dtype, as in ``rope``: computed in float32 with
every product and sum rounded on its own, so that stored bytes can be compared.
"""

import numpy as np

from . import rope
from .numerics import widen

ROPE = 64


def rotate(x, cos, sin, interleaved, dtype):
    """x [..., 64] in storage dtype; pairs (i, i + 32), or (2 i, 2 i + 1) if interleaved."""
    if not interleaved:
        return rope.rotate_storage(x, cos, sin, dtype)
    order = np.concatenate([np.arange(0, ROPE, 2), np.arange(1, ROPE, 2)])
    y = rope.rotate_storage(np.ascontiguousarray(x[..., order]), cos, sin, dtype)
    out = np.empty_like(y)
    out[..., order] = y
    return out


def norm(x, weight, eps):
    """float64 rows [T, R]."""
    return x * weight / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def angles(table, positions):
    cs = table[np.asarray(positions)]
    return cs[:, :ROPE // 2], cs[:, ROPE // 2:]


def append(latent, k_rope, slots, positions, table, block_size, num_blocks, dtype, weight=None,
           eps=1e-6, interleaved=False):
    """(latent part float64 [NB, bs, R], key part in storage dtype [NB, bs, 64], written
    [NB, bs]): what the cache holds after the append, before the norm is rounded."""
    x = widen(latent, dtype)
    if weight is not None:
        x = norm(x, widen(weight, dtype), eps)
    cos, sin = angles(table, positions)
    key = rotate(k_rope, cos, sin, interleaved, dtype)
    a = np.zeros((num_blocks, block_size, latent.shape[1]))
    b = np.zeros((num_blocks, block_size, ROPE), dtype=key.dtype)
    done = np.zeros((num_blocks, block_size), bool)
    for t, s in enumerate(np.asarray(slots)):
        if s < 0:
            continue
        a[s // block_size, s % block_size] = x[t]
        b[s // block_size, s % block_size] = key[t]
        done[s // block_size, s % block_size] = True
    return a, b, done


def rows_of(cache, table, n):
    """The first n cached rows of a sequence, storage dtype [n, R + 64]."""
    bs = cache.shape[1]
    return np.concatenate([cache[int(b)] for b in table[:-(-n // bs)]])[:n] if n else cache[0, :0]


def softmax_rows(x):
    p = np.exp(x - x.max(-1, keepdims=True))
    return p / p.sum(-1, keepdims=True)


def absorbed(q, cache, tables, start, ctx, scale, dtype):
    """q [T, H, R + 64] in storage dtype; float64 out [T, H, R] (rows of no sequence: NaN)."""
    r = cache.shape[2] - ROPE
    out = np.full(q.shape[:2] + (r,), np.nan)
    qf = widen(q, dtype)
    for s, c in enumerate(int(x) for x in ctx):
        rows = widen(rows_of(cache, tables[s], c), dtype)
        m = int(start[s + 1]) - int(start[s])
        for i in range(m):
            n = c - m + i + 1
            p = softmax_rows(qf[start[s] + i] @ rows[:n].T * scale)
            out[start[s] + i] = p @ rows[:n, :r]
    return out


def expanded(q, k, v, k_rope, q_start, k_start, scale, dtype):
    """q [Tq, H, D + 64], k, v [Tk, H, D], k_rope [Tk, 64]; float64 out [Tq, H, D] (rows of
    no sequence: NaN; a query that sees no key: zeros)."""
    d = v.shape[2]
    out = np.full(q.shape[:2] + (d,), np.nan)
    qf, kf, vf, rf = (widen(x, dtype) for x in (q, k, v, k_rope))
    for s in range(len(q_start) - 1):
        a, b, m = int(k_start[s]), int(k_start[s + 1]), int(q_start[s + 1] - q_start[s])
        for i in range(m):
            t, n = int(q_start[s]) + i, b - a - m + i + 1
            if n <= 0:
                out[t] = 0.0
                continue
            x = np.einsum("hd,jhd->hj", qf[t, :, :d], kf[a:a + n]) + qf[t, :, d:] @ rf[a:a + n].T
            out[t] = np.einsum("hj,jhd->hd", softmax_rows(x * scale), vf[a:a + n])
    return out
