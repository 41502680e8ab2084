"""GPU: absorbed attention of batches in which one sequence has many more (token, head) rows
than the others.  The kernel is chosen by a batch's mean, so the rows of a long sequence then
are several tiles of the kernel for few rows."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import latent  # noqa: E402
from tests.latent_checks import absorbed_bound, assert_close  # noqa: E402
from tests.sparse_checks import values  # noqa: E402
from tests.test_gpu_latent import SCALE, attend, batch, pkv  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,r,h,new,ctx,mean", [
    # 320 rows of one sequence, five tiles of 64, over keys that many CTAs share
    ("bf16", 512, 8, [40] + [1] * 9, [3000, 1, 16, 33, 500, 70, 31, 32, 64, 90], 64),
    ("bf16", 128, 8, [1] * 9 + [40], [100, 1, 16, 33, 500, 70, 31, 32, 64, 40], 64),
    # 168 rows: two tiles and a part, a tile's causal limits in front of the last keys
    ("bf16", 256, 24, [7, 1, 1, 1, 1, 1], [2500, 40, 3, 130, 65, 17], 64),
    ("bf16", 384, 24, [1, 7, 1, 0, 2, 1], [20, 7, 600, 9, 2, 33], 64),
    # 33 tokens, more than the keys of a tile: rows that end in front of a stretch
    ("bf16", 512, 3, [33, 1, 1, 1], [33, 2000, 5, 77], 64),
    # single precision: units of 8, 16 and 32 rows, chosen the same way
    ("f32", 256, 2, [20] + [1] * 12, [1500, 1, 2, 3, 40, 50, 60, 70, 80, 16, 17, 31, 33], 8),
    ("f32", 512, 4, [24] + [1] * 9, [1100, 9, 200, 3, 40, 50, 60, 70, 80, 16], 16),
    ("f32", 128, 5, [40, 1, 1], [900, 30, 4], 1 << 20),
])
def test_one_long_sequence_among_short_ones(pkv, dtype, r, h, new, ctx, mean):  # noqa: F811
    rows = -(-sum(new) // len(new)) * h
    assert rows <= mean and max(new) * h > min(mean, 64)
    rng = np.random.default_rng(h)
    cache, t = batch(rng, dtype, r, ctx)
    start = np.concatenate([[0], np.cumsum(new)])
    q = values(rng, (start[-1], h, r + 64), dtype)
    args = (q, cache, t, start, ctx, SCALE, dtype)
    ref = latent.absorbed(*args)
    out, code = attend(pkv, q, cache, t, ctx, dtype, start)
    assert code == 0
    assert_close(out, ref, absorbed_bound(*args, ref))
    again, _ = attend(pkv, q, cache, t, ctx, dtype, start, ws_byte=0x11)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype,r,h", [("bf16", 512, 16), ("bf16", 256, 40), ("f32", 256, 4)])
def test_padding_chooses_another_kernel_and_not_another_result(pkv, dtype, r, h):  # noqa: F811
    """Query rows behind the last sequence count in the mean: the same sequences with and
    without them, both within the bound."""
    rng = np.random.default_rng(h)
    ctx, start = [700, 40, 333], [0, 1, 2, 3]
    cache, t = batch(rng, dtype, r, ctx)
    q = values(rng, (3, h, r + 64), dtype)
    args = (q, cache, t, start, ctx, SCALE, dtype)
    ref = latent.absorbed(*args)
    bound = absorbed_bound(*args, ref)
    for pad in (0, 40):
        nan = np.full((pad, h, r + 64), 0x7FC0 if dtype == "bf16" else np.nan, q.dtype)
        out, code = attend(pkv, np.concatenate([q, nan]), cache, t, ctx, dtype, start)
        assert code == 0
        assert_close(out[:3], ref, bound)
        assert (out[3:] == 7.0).all()
