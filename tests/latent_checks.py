"""Inputs and error bounds shared by the latent-attention tests."""

import numpy as np

from oracle import latent
from oracle.numerics import widen
from tests.gpu_parity import gamma
from tests.sparse_checks import EXP2_REL, ROUND

# half a step of a bf16 weight, relative: P enters the second product in bf16
P_ROUND = {"bf16": 2.0 ** -8, "f32": 0.0}


def latent_cache(rng, nb, r, dtype, fill=None):
    """A pool of NaN (what no token was written to may hold anything)."""
    bits = np.uint16 if dtype == "bf16" else np.float32
    if fill is not None:
        return np.full((nb, 16, r + latent.ROPE), fill, bits)
    return np.full((nb, 16, r + latent.ROPE), 0x7FC1 if dtype == "bf16" else np.nan, bits)


def fill(cache, table, rows):
    """Write a sequence's rows into its blocks."""
    for i, row in enumerate(rows):
        cache[table[i // 16], i % 16] = row


def _bound(x_abs, scale, p, v, o, n, dims, dtype, same_sum):
    """|kernel - o| for one row, from the arithmetic alone.

    Over n keys with weights p (sum 1), S = scale max_j sum_d |q_d k_jd|, W = sum_j p_j
    |v_j - o|, A = sum_j p_j |v_j|:
      * a score is a dims-term dot product in single precision, scaled, offset and
        exponentiated: each weight is off by gamma_{dims+4} S + 2^-21 relative, which
        moves the output by that times W;
      * a weight rounded to bf16 is off by 2^-8 relative: that times W where the sum of
        weights is taken of the rounded ones (what all share cancels), else times A + |o|;
        where they are subnormal or below, what is lost is below 2^-126 of the sum;
      * numerator and denominator are sums of n terms, each rescaled at most once a term
        and once more for each of up to 152 parts joined; tensor-core sums may cut instead
        of round, which doubles the unit: 2 gamma_{2 n + 304} (A + |o|);
      * the output's own rounding, half a step.
    """
    s = abs(scale) * float(x_abs.max())
    a, w = p @ np.abs(v), p @ np.abs(v - o)
    pr = P_ROUND[dtype] * (1.0 + 2.0 ** -7)
    return ((gamma(dims + 4) * s + EXP2_REL) * w + pr * (w if same_sum else a + np.abs(o))
            + 2 * gamma(2 * n + 304) * (a + np.abs(o)) + ROUND[dtype] * np.abs(o) + 1e-30)


def absorbed_bound(q, cache, tables, start, ctx, scale, dtype, ref):
    r = cache.shape[2] - latent.ROPE
    qf, out = widen(q, dtype), np.zeros_like(ref)
    for s, c in enumerate(int(x) for x in ctx):
        rows = widen(latent.rows_of(cache, tables[s], c), dtype)
        m = int(start[s + 1]) - int(start[s])
        for i in range(m):
            t, n = int(start[s]) + i, c - m + i + 1
            for h in range(q.shape[1]):
                p = latent.softmax_rows((rows[:n] @ qf[t, h] * scale)[None])[0]
                out[t, h] = _bound(np.abs(rows[:n]) @ np.abs(qf[t, h]), scale, p, rows[:n, :r],
                                   ref[t, h], n, r + latent.ROPE, dtype, True)
    return out


def expanded_bound(q, k, v, k_rope, q_start, k_start, scale, dtype, ref):
    d = v.shape[2]
    qf, kf, vf, rf = (widen(x, dtype) for x in (q, k, v, k_rope))
    out = np.zeros_like(ref)
    for s in range(len(q_start) - 1):
        a, b, m = int(k_start[s]), int(k_start[s + 1]), int(q_start[s + 1] - q_start[s])
        for i in range(m):
            t, n = int(q_start[s]) + i, b - a - m + i + 1
            if n <= 0:
                continue
            for h in range(q.shape[1]):
                keys = np.concatenate([kf[a:a + n, h], rf[a:a + n]], axis=1)
                p = latent.softmax_rows((keys @ qf[t, h] * scale)[None])[0]
                out[t, h] = _bound(np.abs(keys) @ np.abs(qf[t, h]), scale, p, vf[a:a + n, h],
                                   ref[t, h], n, d + latent.ROPE, dtype, False)
    return out


def assert_close(got, ref, bound):
    got = got.float().cpu().numpy().astype(np.float64)
    live = np.isfinite(ref)
    assert np.isfinite(got[live]).all()
    over = (np.abs(got - ref) - bound)[live]
    assert over.max() <= 0.0, (over.max(), np.abs(got - ref)[live].max())
