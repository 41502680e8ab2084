"""GPU: offsets that do not fit, in the attention over latent caches and over expanded keys:
which rows are computed, which are left as they were, and what is flagged."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import latent  # noqa: E402
from tests.latent_checks import absorbed_bound, assert_close, expanded_bound  # noqa: E402
from tests.sparse_checks import i32, to_dev, values  # noqa: E402
from tests.test_gpu_expanded import Case  # noqa: E402
from tests.test_gpu_latent import SCALE, attend, batch, pkv  # noqa: E402, F401

pytestmark = pytest.mark.gpu

BAD_LAYOUT = 5


@pytest.mark.parametrize("dtype,h", [("bf16", 3), ("bf16", 90), ("f32", 3), ("f32", 40)])
@pytest.mark.parametrize("start,live", [
    ([0, 2, 1, 3], {0: (0, 0), 2: (2, 1)}),       # the second falls; row 1 has two owners
    ([1, 2, 3, 4], {2: (1, 0), 3: (2, 0)}),       # the first does not begin with 0
    ([0, 1, 2, 9], {0: (0, 0), 1: (1, 0)}),       # the last ends behind the call's rows
    ([0, -1, 2, 3], {2: (2, 0)}),                 # the first falls, the second begins below 0
])
def test_latent_offsets(pkv, dtype, h, start, live):  # noqa: F811
    """live: row -> (sequence, its token) of the rows that a sequence in order holds alone."""
    rng = np.random.default_rng(15)
    ctx = [40, 150, 60]
    cache, t = batch(rng, dtype, 128, ctx)
    q = values(rng, (4, h, 192), dtype)
    out, code = attend(pkv, q, cache, t, ctx, dtype, start)
    assert code == BAD_LAYOUT
    named = {r for s in range(3) if start[s] == 0 or s > 0 for r in range(max(0, start[s]), start[s + 1])
             if start[s] >= 0 and start[s + 1] <= 4}
    for row in range(4):
        if row not in named:
            assert (out[row] == 7.0).all(), row
    for row, (s, i) in live.items():
        m = start[s + 1] - start[s]
        # token i of m sees keys 0 .. ctx - m + i
        args = (q[row:row + 1], cache, t[s:s + 1], [0, 1], [ctx[s] - m + i + 1], SCALE, dtype)
        ref = latent.absorbed(*args)
        assert_close(out[row:row + 1], ref, absorbed_bound(*args, ref))


@pytest.mark.parametrize("dtype,keys", [("bf16", 30), ("bf16", 1200), ("f32", 30)])
@pytest.mark.parametrize("q_start,k_start,live", [
    ([0, 20, 10, 60], None, [0]),                 # (the last begins inside the first)
    ([0, 20, 40, 200], None, [0, 1]),
    (None, [0, 1, -10, 3], [0]),
    (None, [0, 1, 2, 900], [0, 1]),
    ([1, 20, 40, 60], None, [1, 2]),
    (None, [-1, 1, 2, 3], [1, 2]),
])
def test_expanded_offsets(pkv, dtype, keys, q_start, k_start, live):  # noqa: F811
    """Key offsets in units of a sequence's keys; the longer ones in clusters."""
    c = Case(np.random.default_rng(5), dtype, 2, 128, [20, 20, 20], [keys] * 3, pad=0)
    ks = None if k_start is None else [k * keys if k > 0 else k for k in k_start]
    out, code = c.run(pkv, q_start=q_start, k_start=ks)
    assert code == BAD_LAYOUT
    if q_start is not None:
        c.qs = np.array(q_start)
    if ks is not None:
        c.ks = np.array(ks)
    for s in range(3):
        a, b = c.qs[s], c.qs[s + 1]
        if s in live:
            args = (c.q[a:b], np.ascontiguousarray(c.kv[c.ks[s]:c.ks[s + 1], :, :128]),
                    np.ascontiguousarray(c.kv[c.ks[s]:c.ks[s + 1], :, 128:]), c.r[c.ks[s]:c.ks[s + 1]],
                    [0, b - a], [0, c.ks[s + 1] - c.ks[s]], c.scale, dtype)
            ref = latent.expanded(*args)
            bound = expanded_bound(*args, ref)
            own = slice(0, 10) if q_start == [0, 20, 10, 60] else slice(None)   # rows of its own
            assert_close(out[a:b][own], ref[own], bound[own])
        elif q_start != [0, 20, 10, 60]:
            rows = range(max(0, a), min(b, 60))
            assert (out[list(rows)] == 7.0).all(), s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expanded_bound_of_no_queries(pkv, dtype):  # noqa: F811
    """A bound of 0 queries a sequence: longer ones are flagged as for any other bound."""
    c = Case(np.random.default_rng(6), dtype, 2, 64, [3, 0, 2], [5, 4, 2], pad=0)
    q, kv, r = (to_dev(x, dtype) for x in (c.q, c.kv, c.r))
    out = torch.full((5, 2, 64), 7.0, dtype=q.dtype, device="cuda")
    pkv.pkv_attention_expanded(out, q, kv[..., :64], kv[..., 64:], r, i32(c.qs), i32(c.ks), 0)
    assert pkv.device_error() == BAD_LAYOUT and (out == 7.0).all()
    pkv.pkv_attention_expanded(out, q, kv[..., :64], kv[..., 64:], r, i32([0, 0, 0, 0]), i32(c.ks), 0)
    assert pkv.device_error() == 0 and (out == 7.0).all()
