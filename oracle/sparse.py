"""Device block tables, key bounds, block selection and sparse attention (oracle).

Written from the definitions, request by request and block by block, in float64
and Python integers:

  * a step of the device block tables is what a pool with a stack of free ids
    does for the requests one after the other [Deploy §2.1 3. (blocks taken when
    the last one is full); Infra 二 (free block list)];
  * the bounds of a (block, KV head) are the largest and the smallest key value
    of each dimension, rounded outwards to whole multiples of 2^e, e the least
    exponent with max |k| <= 127 * 2^e within -50 .. 50;
  * a block scores max over the group's heads of sum_d max(q_d hi_d, q_d lo_d)
    with the query rounded to multiples of its own 2^f.  All values are small
    integers times powers of two, so float64 is exact;
  * sparse attention is softmax(q K^T * scale) V over the keys of the listed
    blocks that the row sees [Ch15 §15.1], each listed block counted as often as
    it is listed; a row that sees no listed key is 0.
"""

import math

import numpy as np

from .numerics import widen


# ---- block tables ------------------------------------------------------------
class TablesModel:
    """Block tables and a stack of free ids, served request by request."""

    def __init__(self, num_blocks, block_size, max_seqs, max_blocks, order=None):
        self.bs, self.num_blocks = block_size, num_blocks
        self.table = np.full((max_seqs, max_blocks), -1, dtype=np.int64)
        order = list(range(num_blocks)) if order is None else [int(b) for b in order]
        self.free = order[::-1]

    def step(self, rows, cached, new, max_tokens, width):
        """Returns (context_lens, query_start_loc, slots, positions, tables)."""
        n, bs = len(cached), self.bs
        rows = list(range(n)) if rows is None else [int(r) for r in rows]
        new = [1] * n if new is None else [int(x) for x in new]
        ctx, start = [], [0]
        slots, pos = [], []
        tables = np.full((n, width), -1, dtype=np.int64)
        full = False
        for i, r in enumerate(rows):
            total = int(cached[i]) + new[i]
            ok = (0 <= r < self.table.shape[0] and rows.count(r) == 1 and cached[i] >= 0
                  and new[i] >= 0 and total <= min(width, self.table.shape[1]) * bs)
            if not ok:
                ctx.append(0)
                start.append(start[-1])
                continue
            need = -(-total // bs) - -(-int(cached[i]) // bs)
            full = full or need > len(self.free) or start[-1] + new[i] > max_tokens
            if full:
                total = int(cached[i])
            for b in range(-(-int(cached[i]) // bs), -(-total // bs)):
                self.table[r, b] = self.free.pop()
            for p in range(int(cached[i]), total):
                slots.append(int(self.table[r, p // bs]) * bs + p % bs)
                pos.append(p)
            blocks = -(-total // bs)
            tables[i, :blocks] = self.table[r, :blocks]
            ctx.append(total)
            start.append(len(slots))
        pad = max_tokens - len(slots)
        return (np.array(ctx, dtype=np.int64), np.array(start), np.array(slots + [-1] * pad),
                np.array(pos + [0] * pad), tables)

    def release(self, rows, lens):
        for r, n in zip(rows, lens):
            blocks = -(-int(n) // self.bs)
            self.free.extend(int(b) for b in self.table[r, :blocks])
            self.table[r, :blocks] = -1


# ---- bounds and selection ------------------------------------------------------
def exponent(amax):
    """The least e of -50 .. 50 with amax <= 127 * 2^e (50 if there is none)."""
    e = -50
    while e < 50 and amax > 127.0 * 2.0 ** e:
        e += 1
    return e


def block_bounds(keys):
    """keys float64 [rows, D] of one (block, head): (codes [2, D], e)."""
    if not np.isfinite(keys).all():
        return np.zeros((2, keys.shape[1]), dtype=np.int64), 127
    e = exponent(np.abs(keys).max())
    hi, lo = keys.max(0) / 2.0 ** e, keys.min(0) / 2.0 ** e
    return np.clip(np.stack([np.ceil(hi), np.floor(lo)]), -127, 127).astype(np.int64), e


def update_bounds(bounds, exps, k_cache, block_tables, query_start_loc, context_lens, dtype):
    """In place, for the blocks that hold each sequence's last qlen positions."""
    bs = k_cache.shape[2]
    for s, ctx in enumerate(int(c) for c in context_lens):
        q = int(query_start_loc[s + 1]) - int(query_start_loc[s])
        if q == 0:
            continue
        for b in range((ctx - q) // bs, -(-ctx // bs)):
            blk = int(block_tables[s, b])
            rows = min(bs, ctx - b * bs)
            for h in range(k_cache.shape[1]):
                bounds[blk, h], exps[blk, h] = block_bounds(widen(k_cache[blk, h, :rows], dtype))


def row_layout(query_start_loc, context_lens):
    """[(row, sequence, keys the row sees)] of every query row."""
    out = []
    for s, ctx in enumerate(int(c) for c in context_lens):
        r0, r1 = int(query_start_loc[s]), int(query_start_loc[s + 1])
        out += [(r, s, ctx - (r1 - r) + 1) for r in range(r0, r1)]
    return out


def q_codes(q):
    """q float64 [D]: its value rounded to multiples of 2^f."""
    if not np.isfinite(q).all():
        return np.zeros_like(q)
    unit = 2.0 ** exponent(np.abs(q).max())
    return np.clip(np.rint(q / unit), -127, 127) * unit


def block_scores(q, bounds, exps, ids):
    """q float64 [G, D] (one KV head's group), ids the physical blocks; their scores."""
    out = np.full(len(ids), -np.inf)
    codes = [q_codes(x) for x in q]
    for i, b in enumerate(int(x) for x in ids):
        if b < 0 or b >= bounds.shape[0]:
            continue
        if exps[b] == 127:
            out[i] = np.inf
            continue
        ends = bounds[b].astype(np.float64) * 2.0 ** int(exps[b])
        out[i] = max(np.maximum(x * ends[0], x * ends[1]).sum() for x in codes)
    return out


def select(q, bounds, exps, block_tables, query_start_loc, context_lens, block_size, top_k,
           sink, recent, dtype):
    """int [T, Hkv, top_k] (rows that belong to no sequence: -1)."""
    T, hq, _ = q.shape
    hkv = exps.shape[1]
    g = hq // hkv
    qf = widen(q, dtype)
    out = np.full((T, hkv, top_k), -1, dtype=np.int64)
    for r, s, keys in row_layout(query_start_loc, context_lens):
        n = -(-keys // block_size)
        for h in range(hkv):
            ids = block_tables[s, :n]
            sc = block_scores(qf[r, h * g:(h + 1) * g], bounds[:, h], exps[:, h], ids)
            always = [b for b in range(n) if b < sink or b >= n - recent]
            rest = sorted((b for b in range(n) if b not in set(always)),
                          key=lambda b: (-sc[b], b))
            took = sorted(always + rest[:max(0, min(n, top_k) - len(always))])
            out[r, h, :len(took)] = took
    return out


# ---- attention -----------------------------------------------------------------
def attention(q, k_cache, v_cache, block_tables, query_start_loc, context_lens, selected, dtype,
              scale=None):
    """float64 [T, Hq, D] (rows that belong to no sequence: NaN)."""
    T, hq, d = q.shape
    hkv, bs = k_cache.shape[1], k_cache.shape[2]
    g = hq // hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    qf = widen(q, dtype)
    out = np.full((T, hq, d), np.nan)
    for r, s, keys in row_layout(query_start_loc, context_lens):
        for h in range(hkv):
            ks, vs = [], []
            for b in (int(x) for x in selected[r, h]):
                if b < 0 or b * bs >= keys:
                    continue
                rows = min(bs, keys - b * bs)
                blk = int(block_tables[s, b])
                ks.append(widen(k_cache[blk, h, :rows], dtype))
                vs.append(widen(v_cache[blk, h, :rows], dtype))
            if not ks:
                out[r, h * g:(h + 1) * g] = 0.0
                continue
            k, v = np.concatenate(ks), np.concatenate(vs)
            x = (qf[r, h * g:(h + 1) * g] @ k.T) * scale
            p = np.exp(x - x.max(axis=1, keepdims=True))
            out[r, h * g:(h + 1) * g] = (p @ v) / p.sum(axis=1, keepdims=True)
    return out
