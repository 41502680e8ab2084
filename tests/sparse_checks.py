"""Inputs and error bounds shared by the sparse-attention tests."""

import math

import numpy as np
import torch

from oracle import sparse
from oracle.numerics import widen
from tests.gpu_parity import gamma

EXP2_REL = 2.0 ** -21      # relative error allowed for exp2 in single precision (a few ulps)
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}    # half a step of the output type, relative


def to_dev(a, dtype=None, device="cuda"):
    """A storage array (uint16 bf16 bits, float32 or integers) as a device tensor."""
    a = np.ascontiguousarray(a)
    if dtype == "bf16":
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
    return torch.from_numpy(a).to(device)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def values(rng, shape, dtype, scale=1.0):
    x = (rng.standard_normal(shape) * scale).astype(np.float32)
    if dtype == "f32":
        return x
    return (x.view(np.uint32) >> 16).astype(np.uint16)     # towards zero: any bf16 value serves


def tables_for(rng, ctx, bs=16, slack=5, width=None):
    """(block tables padded with -1, pool size) over a shuffled pool."""
    blocks = [-(-int(c) // bs) for c in ctx]
    nb = sum(blocks) + slack
    ids = rng.permutation(nb)
    t = np.full((len(ctx), width or max(blocks)), -1, dtype=np.int32)
    at = 0
    for s, n in enumerate(blocks):
        t[s, :n] = ids[at:at + n]
        at += n
    return t, nb


def attention_bound(q, k_cache, v_cache, block_tables, start, ctx, selected, dtype, ref,
                    scale=None):
    """Element-wise bound of |kernel - ref|, from the arithmetic alone.

    Over the n keys a row sees, with weights p (sum 1), exact output o, and
      S = scale * max_j sum_d |q_d k_jd|,  W_d = sum_j p_j |v_jd - o_d|,
      A_d = sum_j p_j |v_jd|:
      * a score is a D-term dot product in single precision, scaled and offset,
        and exponentiated: each weight is off by at most gamma_{D+4} S + 2^-21
        relative, which moves the output by that times W;
      * in the product with V a weight may stand as the sum of two bf16 values:
        the first leaves at most 2^-8 of it, the second at most 2^-8 of that:
        2^-16 A;
      * numerator and denominator are sums of n terms, rescaled at most once
        for each of them: at most gamma_{2n} each, and tensor-core sums may cut
        instead of round, which doubles the unit: 2 gamma_{2n} (A + |o|);
      * the output's own rounding, half a step: ROUND |o|.
    """
    g = q.shape[1] // k_cache.shape[1]
    d, bs = q.shape[2], k_cache.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    qf = widen(q, dtype)
    bound = np.zeros_like(ref)
    for r, s, keys in sparse.row_layout(start, ctx):
        for h in range(k_cache.shape[1]):
            ks, vs = [], []
            for b in (int(x) for x in selected[r, h]):
                if b < 0 or b * bs >= keys:
                    continue
                rows, blk = min(bs, keys - b * bs), int(block_tables[s, b])
                ks.append(widen(k_cache[blk, h, :rows], dtype))
                vs.append(widen(v_cache[blk, h, :rows], dtype))
            if not ks:
                continue
            k, v = np.concatenate(ks), np.concatenate(vs)
            n = k.shape[0]
            for j in range(h * g, (h + 1) * g):
                x = (k @ qf[r, j]) * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                S = abs(scale) * float((np.abs(k) @ np.abs(qf[r, j])).max())
                A, o = p @ np.abs(v), ref[r, j]
                W = p @ np.abs(v - o)
                bound[r, j] = ((gamma(d + 4) * S + EXP2_REL) * W + 2.0 ** -16 * A
                               + 2 * gamma(2 * n) * (A + np.abs(o)) + ROUND[dtype] * np.abs(o)
                               + 1e-30)
    return bound


def assert_attention(out, ref, bound):
    got = out.float().cpu().numpy().astype(np.float64)
    live = np.isfinite(ref)
    assert np.isfinite(got[live]).all()
    over = np.abs(got - ref)[live] - bound[live]
    assert over.max() <= 0.0, (over.max(), np.abs(got - ref)[live].max())
