"""GPU: infinite scores in the attention over latent caches and over expanded keys, in every
form that the calls take: a key whose score is -inf weighs nothing, and a query all of whose
scores are -inf has no weights, so that its output is 0 / 0."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import latent  # noqa: E402
from oracle.numerics import widen  # noqa: E402
from tests.latent_checks import absorbed_bound, assert_close, expanded_bound, fill, latent_cache  # noqa: E402
from tests.sparse_checks import tables_for, values  # noqa: E402
from tests.test_gpu_expanded import Case  # noqa: E402
from tests.test_gpu_latent import SCALE, attend, pkv  # noqa: E402, F401

pytestmark = pytest.mark.gpu

INF = {"bf16": (0x7F80, 0xFF80), "f32": (np.float32(np.inf), np.float32(-np.inf))}


def positive(x, dtype):
    """0.5 or more in magnitude, and above 0."""
    y = np.abs(widen(x, dtype)).astype(np.float32) + np.float32(0.5)
    return y if dtype == "f32" else (y.view(np.uint32) >> 16).astype(np.uint16)


# dtype, heads, queries, keys: one CTA a unit, clusters of four and of two, single precision in
# clusters and alone
FORMS = [("bf16", 2, [40, 30], [200, 290]), ("bf16", 2, [40], [1300]), ("bf16", 50, [20], [1500]),
         ("f32", 2, [40, 30], [200, 290]), ("f32", 110, [180, 20], [400, 90])]


def sampled(c, heads):
    """What the oracle takes of some heads of a case."""
    return (np.ascontiguousarray(c.q[:, heads]), np.ascontiguousarray(c.kv[:, heads, :c.d]),
            np.ascontiguousarray(c.kv[:, heads, c.d:]), c.r, c.qs, c.ks, c.scale, c.dtype)


def without(c, keys):
    """The same case without some of the first sequence's keys."""
    e = Case.__new__(Case)
    e.__dict__.update(c.__dict__)
    e.kv, e.r = np.delete(c.kv, keys, 0), np.delete(c.r, keys, 0)
    e.ks = np.concatenate([[0], c.ks[1:] - len(keys)])
    return e


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,h,new,keys", FORMS)
def test_expanded_keys_of_minus_infinity_weigh_nothing(pkv, dtype, h, new, keys, d):  # noqa: F811
    """Some of the prefix's keys, a whole tile and a whole CTA's share among them: the
    result is that of the call without them."""
    c = Case(np.random.default_rng(h + d), dtype, h, d, new, keys)
    c.q[..., d], c.r[:c.ks[-1], 0] = positive(c.q[..., d], dtype), positive(c.r[:c.ks[-1], 0], dtype)
    n = keys[0] - new[0]
    gone = [j for j in range(n) if j < 130 or j % 7 == 0 or 380 <= j < 770]
    args = sampled(without(c, gone), [0, h - 1])
    ref = latent.expanded(*args)
    bound = expanded_bound(*args, ref)
    c.r[gone, 0] = INF[dtype][1]
    out, code = c.run(pkv)
    assert code == 0
    assert_close(out[:, [0, h - 1]], ref, bound)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,h,new,keys", FORMS)
def test_expanded_queries_whose_scores_are_all_minus_infinity(pkv, dtype, h, new, keys, d):  # noqa: F811
    """NaN for these, whichever form the call takes; the other queries as always."""
    c = Case(np.random.default_rng(h + d), dtype, h, d, new, keys)
    c.r[:c.ks[-1], 0] = positive(c.r[:c.ks[-1], 0], dtype)
    args = sampled(c, [0, h - 1])
    ref = latent.expanded(*args)
    bound = expanded_bound(*args, ref)
    rows = [0, 7, new[0] - 1]
    c.q[rows, :, d] = INF[dtype][1]
    ref[rows] = np.nan
    out, code = c.run(pkv)
    assert code == 0
    assert torch.isnan(out[rows]).all()
    assert_close(out[:, [0, h - 1]], ref, bound)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,h,new,keys", FORMS)
def test_an_infinite_score_is_seen_by_those_queries_alone_that_see_its_key(pkv, dtype, h, new, keys, d):  # noqa: F811
    """+inf leaves no weights either (inf - inf); queries in front of the key are as always."""
    c = Case(np.random.default_rng(h + d), dtype, h, d, new, keys)
    c.q[..., d] = positive(c.q[..., d], dtype)
    args = sampled(c, [0, h - 1])
    ref = latent.expanded(*args)
    bound = expanded_bound(*args, ref)
    c.r[keys[0] - 5, 0] = INF[dtype][0]
    ref[new[0] - 5:new[0]] = np.nan
    out, code = c.run(pkv)
    assert code == 0
    assert torch.isnan(out[new[0] - 5:new[0]]).all()
    assert_close(out[:, [0, h - 1]], ref, bound)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,new,keys,bad", [(2, [16, 9, 11], [1500, 900, 1000], 1),
                                            (14, [16, 9, 30], [1200, 1100, 1300], 0)])
def test_a_neighbours_nan_does_not_reach_a_cluster(pkv, d, h, new, keys, bad):  # noqa: F811
    """Units shared by four CTAs and by two, whose last tiles hold the next sequence's rows."""
    c = Case(np.random.default_rng(h + d), "bf16", h, d, new, keys)
    args = sampled(c, [0, h - 1])
    ref = latent.expanded(*args)
    bound = expanded_bound(*args, ref)
    rows, own = slice(c.ks[bad], c.ks[bad + 1]), slice(c.qs[bad], c.qs[bad + 1])
    c.kv[rows], c.r[rows] = 0x7FC0, 0x7FC0
    ref[own] = np.nan
    out, code = c.run(pkv)
    assert code == 0 and torch.isnan(out[own]).all()
    assert_close(out[:, [0, h - 1]], ref, bound)


CACHES = [("bf16", 8, 128), ("bf16", 90, 128), ("bf16", 24, 512), ("bf16", 128, 512), ("f32", 8, 256)]


@pytest.mark.parametrize("dtype,h,r", CACHES)
def test_cached_rows_of_minus_infinity_weigh_nothing(pkv, dtype, h, r):  # noqa: F811
    """Stretches longer than a CTA's share, and single rows; two query tokens a sequence."""
    rng = np.random.default_rng(h)
    ctx, new = [6000, 300, 40], [2, 2, 2]
    gone = [*range(100), *range(2000, 4000), *range(4001, 5900, 9)]
    q = values(rng, (6, h, r + 64), dtype)
    q[..., r] = positive(q[..., r], dtype)
    rows = [values(rng, (n, r + 64), dtype) for n in ctx]
    for x in rows:
        x[:, r] = positive(x[:, r], dtype)
    t, nb = tables_for(rng, ctx)
    cache, less = latent_cache(rng, nb, r, dtype), latent_cache(rng, nb, r, dtype)
    for s, x in enumerate(rows):
        fill(less, t[s], np.delete(x, gone, 0) if s == 0 else x)
        if s == 0:
            x[gone, r] = INF[dtype][1]
        fill(cache, t[s], x)
    start = [0, 2, 4, 6]
    pick = [0, h // 2, h - 1]
    args = (np.ascontiguousarray(q[:, pick]), less, t, start, [6000 - len(gone), 300, 40], SCALE, dtype)
    ref = latent.absorbed(*args)
    out, code = attend(pkv, q, cache, t, ctx, dtype, start)
    assert code == 0
    assert_close(out[:, pick], ref, absorbed_bound(*args, ref))


@pytest.mark.parametrize("dtype,h,r", CACHES)
@pytest.mark.parametrize("n", [50, 5000])
def test_rows_whose_scores_are_all_minus_infinity(pkv, dtype, h, r, n):  # noqa: F811
    """NaN, in whole units and in units that are cut and joined."""
    rng = np.random.default_rng(h)
    ctx = [n, 33, 70]
    q = values(rng, (3, h, r + 64), dtype)
    t, nb = tables_for(rng, ctx)
    cache = latent_cache(rng, nb, r, dtype)
    for s, m in enumerate(ctx):
        x = values(rng, (m, r + 64), dtype)
        x[:, r] = positive(x[:, r], dtype)
        fill(cache, t[s], x)
    pick, start = [0, h - 1], np.arange(4)
    args = (np.ascontiguousarray(q[:, pick]), cache, t, start, ctx, SCALE, dtype)
    ref = latent.absorbed(*args)
    bound = absorbed_bound(*args, ref)
    q[0, :, r] = INF[dtype][1]
    ref[0] = np.nan
    out, code = attend(pkv, q, cache, t, ctx, dtype)
    assert code == 0 and torch.isnan(out[0]).all()
    assert_close(out[:, pick], ref, bound)
