"""GPU: key bounds and scores at the ends of their arithmetic, against the float64
restatement."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sparse  # noqa: E402
from tests.sparse_checks import i32, to_dev  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("large", [1.0, 300.0, 2.0 ** 40, 2.0 ** 57, 3e38])
def test_tiny_keys_beside_large_ones_are_rounded_outwards(pkv, dtype, d, large):
    """A dimension whose keys are far below the block's unit, down to the least
    subnormal: its upper end is 1 where a key is positive, its lower one -1 where a
    key is negative."""
    tiny = [2.0 ** -149 if dtype == "f32" else 2.0 ** -133, 2.0 ** -126, 2.0 ** -110, 2.0 ** -60]
    k = np.zeros((4, 1, 16, d), dtype=np.float32)
    k[:, 0, 2, 0] = large
    k[1, 0, 9, 0] = -large
    for i, x in enumerate(tiny):
        k[:, 0, i, 1 + i] = x                      # zeros below it
        k[:, 0, i, 11 + i] = -x                    # zeros above it
        k[:, 0, :, 21 + i], k[:, 0, :, 31 + i] = x, -x
        k[:, 0, :8, 41 + i], k[:, 0, 8:, 41 + i] = x, -x
    if dtype == "bf16":
        k = (k.view(np.uint32) >> 16).astype(np.uint16)
    t = np.arange(4, dtype=np.int32)[:, None]
    kd = to_dev(k, dtype)
    bounds, exps = np.zeros((4, 1, 2, d), np.int8), np.zeros((4, 1), np.int8)
    b_d, e_d = to_dev(bounds), to_dev(exps)
    pkv.pkv_block_bounds(b_d, e_d, kd, pkv.cache_desc(kd, 1), i32(t), i32([16] * 4))
    assert pkv.device_error() == 0
    sparse.update_bounds(bounds, exps, k, t, np.arange(5), [16] * 4, dtype)
    assert np.array_equal(e_d.cpu().numpy(), exps)
    assert np.array_equal(b_d.cpu().numpy(), bounds)
    assert (bounds[0, 0, 0, 1:5] == 1).all() and (bounds[0, 0, 1, 11:15] == -1).all()


def _select(pkv, dtype, q, bounds, exps, t, ctx, top_k, sink=0, recent=1):
    """(lists of the call, lists of the float64 restatement), one row a sequence."""
    hq, d = q.shape[1:]
    nb, hkv = exps.shape
    qs = q if dtype == "f32" else (q.view(np.uint32) >> 16).astype(np.uint16)
    desc = pkv.CacheDesc(pkv.PKV_F32 if dtype == "f32" else pkv.PKV_BF16, nb, 16, hkv, hq, d)
    sel = torch.full((q.shape[0], hkv, top_k), -9, dtype=torch.int32, device="cuda")
    pkv.pkv_select_blocks(sel, to_dev(qs, dtype), to_dev(bounds), to_dev(exps), desc, i32(t),
                          i32(ctx), int(max(ctx)), sink, recent)
    assert pkv.device_error() == 0
    ref = sparse.select(qs, bounds, exps, t, np.arange(len(ctx) + 1), ctx, 16, top_k, sink, recent,
                        dtype)
    return sel.cpu().numpy(), ref


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("signs", ["same", "opposite", "mixed"])
def test_scores_of_the_largest_codes_are_exact_to_a_unit(pkv, dtype, d, hq, hkv, signs):
    """Codes of 127 of the query on bounds of 127 in every dimension but the last,
    whose query code is 1: the sums are as large as they get (64 * 127 * 1279 on the
    way), and blocks differ by single units of them."""
    rng = np.random.default_rng(d + hq + len(signs))
    n = 300
    unit = 2.0 ** -3
    sign = np.ones((1, hq, d)) if signs != "mixed" else rng.choice([-1.0, 1.0], (1, hq, d))
    q = (sign * 127.0 * unit).astype(np.float32)
    q[:, :, d - 1] = unit
    side = -1 if signs == "opposite" else 1       # ends beyond zero, on the query's other side
    bounds = np.empty((n, hkv, 2, d), np.int8)
    if signs == "mixed":
        bounds[:] = rng.choice([-127, 127], (1, hkv, 2, d))
    else:
        bounds[:] = 127 * side
    bounds[:, :, :, d - 1] = rng.integers(-127, 128, (n, hkv, 1))
    exps = np.full((n, hkv), -4, np.int8)
    t = rng.permutation(n).astype(np.int32)[None, :]
    for top_k in (20, 131):
        got, ref = _select(pkv, dtype, q, bounds, exps, t, [n * 16], top_k)
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("kind", ["spread", "few", "equal"])
@pytest.mark.parametrize("top_k", [30, 4000])
def test_lists_of_rows_too_long_for_registers(pkv, kind, top_k):
    """Rows from a block to more than 8192 of them in one batch (the longest decides how
    all are read), with last warps that hold no block; scores all over the range, of
    few values, or all the same."""
    rng = np.random.default_rng(top_k)
    blocks = [8193, 1, 9000, top_k, top_k + 1, 16500, 1025, 12288]
    ctx = [16 * b - (i % 3) for i, b in enumerate(blocks)]
    nb, d = sum(blocks) + 3, 64
    ids = rng.permutation(nb)
    t, at = np.full((len(blocks), max(blocks)), -1, dtype=np.int32), 0
    for i, b in enumerate(blocks):
        t[i, :b] = ids[at:at + b]
        at += b
    bounds = np.zeros((nb, 1, 2, d), np.int8)
    exps = np.zeros((nb, 1), np.int8)
    if kind == "spread":
        bounds[:, 0] = rng.integers(-127, 128, (nb, 1, d))
        exps[:, 0] = rng.integers(-20, 20, nb)
    elif kind == "few":
        bounds[:, 0, :, 0] = rng.integers(0, 3, (nb, 1))
        exps[rng.integers(0, nb, 5), 0] = 30
    q = rng.choice([0.0, 0.5, 1.0], (len(blocks), 2, d)).astype(np.float32)
    q[:, :, 0] = 1.0
    got, ref = _select(pkv, "f32", q, bounds, exps, t, ctx, top_k, sink=1, recent=2)
    assert np.array_equal(got, ref)
