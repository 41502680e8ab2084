"""Oracle for latent attention: pinned to closed forms, to the other rotary layout, and
absorbed against expanded attention (CPU)."""

import numpy as np
import pytest

from oracle import attention, latent, rope
from tests.sparse_checks import tables_for, values


def test_interleaved_rotation_is_the_half_form_in_another_order():
    rng = np.random.default_rng(1)
    x = values(rng, (5, 3, 64), "f32")
    cos, sin = latent.angles(rope.rope_table(40, 64), [0, 3, 7, 20, 39])
    y = latent.rotate(x, cos[:, None], sin[:, None], True, "f32")
    z = x[..., 0::2] + 1j * x[..., 1::2]
    w = z.astype(np.complex128) * (cos[:, None].astype(np.float64) + 1j * sin[:, None])
    assert np.allclose(y[..., 0::2], w.real, atol=1e-6)
    assert np.allclose(y[..., 1::2], w.imag, atol=1e-6)
    assert np.array_equal(y[0], x[0])              # position 0: the angle is 0
    half = latent.rotate(x, cos[:, None], sin[:, None], False, "f32")
    order = np.concatenate([np.arange(0, 64, 2), np.arange(1, 64, 2)])
    again = latent.rotate(np.ascontiguousarray(x[..., np.argsort(order)]), cos[:, None],
                          sin[:, None], True, "f32")
    assert np.array_equal(again[..., order], half)


def test_norm_of_equal_values_is_the_weight():
    x = np.full((2, 128), -3.0)
    w = np.linspace(0.5, 2.0, 128)
    assert np.allclose(latent.norm(x, w, 0.0), -w[None])
    assert np.allclose(latent.norm(x, w, 7.0), -w[None] * 3.0 / 4.0)


@pytest.mark.parametrize("ctx,new", [([1, 16, 33], [1, 1, 1]), ([20, 5], [4, 5])])
def test_absorbed_equals_expanded(ctx, new):
    """scale (q . W c + b . k) over expanded keys is (W^T q) . c + b . k over the rows."""
    rng = np.random.default_rng(2)
    r, d, h = 128, 64, 3
    tables, nb = tables_for(rng, ctx)
    cache = values(rng, (nb, 16, r + 64), "f32")
    wk, wv = (values(rng, (h, d, r), "f32", r ** -0.5) for _ in range(2))
    start, k_start = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(ctx)])
    q = values(rng, (start[-1], h, d + 64), "f32")
    rows = np.concatenate([latent.rows_of(cache, tables[s], c) for s, c in enumerate(ctx)])
    c64 = rows[:, :r].astype(np.float64)
    k = np.einsum("hdr,tr->thd", wk.astype(np.float64), c64).astype(np.float32)
    v = np.einsum("hdr,tr->thd", wv.astype(np.float64), c64).astype(np.float32)
    want = latent.expanded(q, k, v, np.ascontiguousarray(rows[:, r:]), start, k_start, 0.09, "f32")
    a = np.einsum("hdr,thd->thr", wk.astype(np.float64), q[..., :d])
    qa = np.concatenate([a, q[..., d:]], -1).astype(np.float32)
    o = latent.absorbed(qa, cache, tables, start, ctx, 0.09, "f32")
    got = np.einsum("hdr,thr->thd", wv.astype(np.float64), o)
    assert np.abs(got - want).max() < 2e-6


def test_expanded_without_a_rotary_part_is_plain_attention():
    rng = np.random.default_rng(3)
    t, nb = tables_for(rng, [37])
    k, v = (values(rng, (nb, 2, 16, 64), "f32") for _ in range(2))
    q = values(rng, (1, 2, 64), "f32")
    want = attention.decode(q, k, v, t, np.array([37], np.int32), 16, "f32")
    rows = [np.concatenate([x[b].transpose(1, 0, 2) for b in t[0]])[:37] for x in (k, v)]
    q0 = np.concatenate([q, np.zeros((1, 2, 64), np.float32)], -1)
    got = latent.expanded(q0, rows[0], rows[1], values(rng, (37, 64), "f32"), [0, 1], [0, 37],
                          1.0 / 8.0, "f32")
    assert np.allclose(got, want, atol=1e-12)


def test_rows_that_see_nothing_are_zero():
    rng = np.random.default_rng(4)
    q, k, r = (values(rng, s, "f32") for s in ((4, 1, 128), (2, 1, 64), (2, 64)))
    out = latent.expanded(q, k, k, r, [0, 4], [0, 2], 0.1, "f32")
    assert (out[:2] == 0).all() and np.allclose(out[2, 0], k[0, 0]) and np.isfinite(out).all()


def test_append_places_rows_and_skips_padding():
    rng = np.random.default_rng(5)
    x, k = values(rng, (4, 128), "bf16"), values(rng, (4, 64), "bf16")
    a, b, done = latent.append(x, k, [17, -1, 0, 3], [0, 5, 0, 2], rope.rope_table(8, 64), 16, 2,
                               "bf16")
    assert done.sum() == 3 and done[1, 1] and done[0, 0] and done[0, 3]
    assert np.array_equal(a[1, 1], latent.widen(x, "bf16")[0]) and np.array_equal(b[1, 1], k[0])
