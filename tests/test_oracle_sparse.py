"""Oracle for the device tables, key bounds, block selection and sparse attention:
pinned to the pool model, to brute force and to the dense oracle (CPU)."""

import numpy as np
import pytest

from oracle import attention, sparse
from oracle.block_pool import OK, BlockPoolModel
from tests.sparse_checks import tables_for, values


@pytest.mark.parametrize("bs", [1, 4, 16])
def test_tables_model_hands_out_the_pools_blocks(bs):
    """Steps and releases give the slots and tables of a pool without sharing."""
    rng = np.random.default_rng(bs)
    nb, rows = 90, 12
    order = rng.permutation(nb)
    pool, model = BlockPoolModel(nb, bs, 0, order), sparse.TablesModel(nb, bs, rows, nb, order)
    lens = [0] * rows
    for _ in range(60):
        n = int(rng.integers(1, rows + 1))
        pick = [int(r) for r in rng.permutation(rows)[:n]]
        new = [int(rng.integers(1, 3 * bs + 2)) for _ in pick]
        need = sum(-(-(lens[r] + x) // bs) - -(-lens[r] // bs) for r, x in zip(pick, new))
        if need > len(model.free):
            live = [r for r in range(rows) if lens[r]]
            model.release(live, [lens[r] for r in live])
            for r in live:
                pool.free_sequence(r)
                lens[r] = 0
            assert model.free[::-1] == [] or len(model.free) == pool.num_free()
            continue
        ctx, start, slots, pos, tables = model.step(pick, [lens[r] for r in pick], new, sum(new),
                                                    nb)
        want = []
        for r, x in zip(pick, new):
            if lens[r] == 0:
                st, got = pool.add_sequence(r, x)
                assert st == OK
                want += got
            else:
                want += [pool.append_slot(r)[0] for _ in range(x)]
            lens[r] += x
        assert slots.tolist() == want and ctx.tolist() == [lens[r] for r in pick]
        assert start.tolist() == np.concatenate([[0], np.cumsum(new)]).tolist()
        for i, r in enumerate(pick):
            t = pool.block_table(r)
            assert tables[i, :len(t)].tolist() == t and (tables[i, len(t):] == -1).all()


def test_exponent_is_the_least_that_holds():
    for e in (-50, -7, 0, 3, 49):
        assert sparse.exponent(127.0 * 2.0 ** e) == e
        assert sparse.exponent(np.nextafter(127.0 * 2.0 ** e, np.inf)) == e + 1
    assert sparse.exponent(0.0) == -50 and sparse.exponent(1e300) == 50


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bounds_hold_every_key_and_scores_bound_every_product(dtype):
    rng = np.random.default_rng(3)
    ctx = [45, 16, 1]
    start = [0, 45, 61, 62]
    t, nb = tables_for(rng, ctx)
    k = values(rng, (nb, 2, 16, 64), dtype, 0.7)
    bounds, exps = np.zeros((nb, 2, 2, 64), np.int64), np.zeros((nb, 2), np.int64)
    sparse.update_bounds(bounds, exps, k, t, start, ctx, dtype)
    q = rng.standard_normal((2, 64))
    for s, c in enumerate(ctx):
        for b in range(-(-c // 16)):
            blk, rows = int(t[s, b]), min(16, c - 16 * b)
            for h in range(2):
                kf = sparse.widen(k[blk, h, :rows], dtype)
                unit = 2.0 ** int(exps[blk, h])
                assert (kf <= bounds[blk, h, 0] * unit).all()
                assert (kf >= bounds[blk, h, 1] * unit).all()
                # less than a unit above what is needed, and no coarser unit than needed
                assert (bounds[blk, h, 0] * unit - kf.max(0) < unit).all()
                assert np.abs(kf).max() > 63.0 * unit
                qr = np.stack([sparse.q_codes(x) for x in q])
                sc = sparse.block_scores(q, bounds[:, h], exps[:, h], [blk])[0]
                assert sc >= (qr @ kf.T).max()


def test_selection_keeps_ends_and_breaks_ties_low():
    nb, hkv, d = 12, 1, 64
    bounds = np.zeros((nb, hkv, 2, d), np.int64)
    bounds[:, :, :, 0] = 5                    # all blocks score alike
    bounds[7, :, :, 0] = 9                    # but one
    exps = np.zeros((nb, hkv), np.int64)
    q = np.zeros((1, 1, d), np.float32)
    q[0, 0, 0] = 1.0
    t = np.arange(nb)[None, :].astype(np.int32)
    got = sparse.select(q, bounds, exps, t, [0, 1], [12 * 16 - 3], 16, 6, 1, 2, "f32")
    assert got[0, 0].tolist() == [0, 1, 2, 7, 10, 11]
    got = sparse.select(q, bounds, exps, t, [0, 1], [5 * 16], 16, 6, 1, 2, "f32")
    assert got[0, 0].tolist() == [0, 1, 2, 3, 4, -1]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_all_blocks_listed_is_dense_attention(dtype):
    rng = np.random.default_rng(5)
    ctx, q_lens = [37, 64, 3], [1, 4, 3]
    start = np.concatenate([[0], np.cumsum(q_lens)])
    t, nb = tables_for(rng, ctx)
    k, v = (values(rng, (nb, 2, 16, 64), dtype) for _ in range(2))
    q = values(rng, (int(start[-1]), 4, 64), dtype)
    sel = np.full((int(start[-1]), 2, 6), -1)
    for r, s, keys in sparse.row_layout(start, ctx):
        n = -(-keys // 16)
        sel[r, :, :n] = rng.permutation(n)
    got = sparse.attention(q, k, v, t, start, ctx, sel, dtype)
    ref = attention.varlen(q, k, v, t, start, ctx, 16, dtype)
    assert np.abs(got - ref).max() < 1e-12
