"""GPU: key bounds and block selection (exact) and attention over listed blocks
(derived bounds), each against its float64 restatement, and a whole step of them."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import attention as oatt  # noqa: E402
from oracle import cache as ocache  # noqa: E402
from oracle import sparse  # noqa: E402
from tests.sparse_checks import (assert_attention, attention_bound, i32, tables_for,  # noqa: E402
                                 to_dev, values)

pytestmark = pytest.mark.gpu

NAN_BITS = np.uint16(0x7FC0)


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


def _poison(cache, tables, ctx, dtype, bs=16):
    """NaN in every row of the pool that holds no token."""
    held = np.zeros((cache.shape[0], bs), dtype=bool)
    for s, c in enumerate(ctx):
        for b in range(-(-int(c) // bs)):
            held[tables[s, b], :min(bs, int(c) - b * bs)] = True
    bad = np.float32(np.nan) if dtype == "f32" else NAN_BITS
    cache.transpose(0, 2, 1, 3)[~held] = bad
    return cache


# ---- bounds -------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,d,ctx,qlen,layout", [
    (8, 128, [1, 16, 17, 700, 31], [1] * 5, False),
    (5, 64, [1, 16, 17, 700, 31], [1] * 5, True),
    (2, 128, [40, 300, 3, 16, 129], [40, 33, 0, 16, 2], True),
    (1, 64, [1500], [1500], True),
    (3, 64, [2100] + [5] * 700, [2000] + [1] * 700, True),
])
def test_bounds_are_exact(pkv, dtype, hkv, d, ctx, qlen, layout):
    rng = np.random.default_rng(hkv * d + len(ctx))
    start = np.concatenate([[0], np.cumsum(qlen)])
    t, nb = tables_for(rng, ctx)
    k = values(rng, (nb, hkv, 16, d), "f32", 1.0) * np.exp2(
        rng.integers(-30, 30, (nb, hkv, 1, 1))).astype(np.float32)
    k[rng.random((nb, hkv)) < 0.1] = 0.0
    if dtype == "bf16":
        k = (k.view(np.uint32) >> 16).astype(np.uint16)
    _poison(k, t, ctx, dtype)
    bounds = np.full((nb, hkv, 2, d), 99, dtype=np.int8)
    exps = np.full((nb, hkv), 99, dtype=np.int8)
    b_d, e_d = to_dev(bounds), to_dev(exps)
    kd = to_dev(k, dtype)
    pad = 3 if layout else 0                       # rows behind the last sequence
    pkv.pkv_block_bounds(b_d, e_d, kd, pkv.cache_desc(kd, hkv), i32(t), i32(ctx),
                         query_start_loc=i32(start) if layout else None,
                         num_query_tokens=int(start[-1]) + pad)
    assert pkv.device_error() == 0
    sparse.update_bounds(bounds, exps, k, t, start, ctx, dtype)
    assert np.array_equal(e_d.cpu().numpy(), exps)
    assert np.array_equal(b_d.cpu().numpy(), bounds)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bounds_at_the_ends_of_the_range(pkv, dtype):
    """Keys that are not finite, huge, tiny, or exactly at a unit's edge."""
    d, special = 64, [np.inf, -np.inf, np.nan, 3e38, 2.0 ** -140, 127.0, 127.0 * 2.0 ** -50,
                      2.0 ** 57, -0.0, 128.0]
    k = np.zeros((len(special), 1, 16, d), dtype=np.float32)
    for i, x in enumerate(special):
        k[i, 0, 3, 5] = x
        k[i, 0, 2, 6] = 0.25
    if dtype == "bf16":
        k = (k.view(np.uint32) >> 16).astype(np.uint16)
    t = np.arange(len(special), dtype=np.int32)[:, None]
    ctx = [16] * len(special)
    kd = to_dev(k, dtype)
    bounds, exps = np.zeros((len(special), 1, 2, d), np.int8), np.zeros((len(special), 1), np.int8)
    b_d, e_d = to_dev(bounds), to_dev(exps)
    pkv.pkv_block_bounds(b_d, e_d, kd, pkv.cache_desc(kd, 1), i32(t), i32(ctx))
    assert pkv.device_error() == 0
    sparse.update_bounds(bounds, exps, k, t, np.arange(len(special) + 1), ctx, dtype)
    assert np.array_equal(e_d.cpu().numpy(), exps)
    assert np.array_equal(b_d.cpu().numpy(), bounds)


def test_bounds_flag_bad_batches(pkv):
    kd = torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    desc = pkv.cache_desc(kd, 1)
    b = torch.full((4, 1, 2, 64), 7, dtype=torch.int8, device="cuda")
    e = torch.full((4, 1), 7, dtype=torch.int8, device="cuda")
    for t, ctx, start, code in (([[4]], [5], None, 1), ([[-1]], [5], None, 1),
                                ([[0]], [17], None, 7), ([[0]], [0], None, 2),
                                ([[0]], [2], [0, 3], 2), ([[0], [1]], [9, 9], [2, 1, 3], 5)):
        n = 3 if start else 1
        pkv.pkv_block_bounds(b, e, kd, desc, i32(t), i32(ctx),
                             query_start_loc=None if start is None else i32(start),
                             num_query_tokens=n)
        assert pkv.device_error() == code
        if code != 5:
            assert (b == 7).all() and (e == 7).all()


# ---- selection -----------------------------------------------------------------
def _select_case(rng, dtype, hq, hkv, d, ctx, qlen, kind="random"):
    t, nb = tables_for(rng, ctx)
    mid = rng.normal(0, 25, (nb, hkv, d))
    half = np.abs(rng.normal(30, 8, (nb, hkv, d)))
    bounds = np.clip(np.rint(np.stack([mid + half, mid - half], 2)), -127, 127).astype(np.int8)
    exps = rng.integers(-7, -4, (nb, hkv)).astype(np.int8)
    if kind == "ties":                             # two kinds of block: most scores are equal
        bounds[:] = bounds[:1]
        exps[:] = -6
        exps[rng.random(nb) < 0.3] = -5
    rows = int(sum(qlen))
    q = values(rng, (rows, hq, d), dtype)
    return t, nb, bounds, exps, q, np.concatenate([[0], np.cumsum(qlen)])


def _run_select(pkv, dtype, q, bounds, exps, t, ctx, start, top_k, sink, recent, max_ctx=None,
                pad=0, layout=True):
    hq, d = q.shape[1:]
    nb, hkv = exps.shape
    desc = pkv.CacheDesc(pkv.PKV_F32 if dtype == "f32" else pkv.PKV_BF16, nb, 16, hkv, hq, d)
    qp = np.concatenate([q, np.zeros((pad, hq, d), q.dtype)])
    sel = torch.full((qp.shape[0], hkv, top_k), -9, dtype=torch.int32, device="cuda")
    pkv.pkv_select_blocks(sel, to_dev(qp, dtype), to_dev(bounds), to_dev(exps), desc, i32(t),
                          i32(ctx), max_ctx or int(max(ctx)), sink, recent,
                          query_start_loc=i32(start) if layout else None)
    got = sel.cpu().numpy()
    assert (got[q.shape[0]:] == -9).all()          # rows behind the last sequence
    return got[:q.shape[0]]


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 8, 128), ("bf16", 8, 4, 64),
                                            ("f32", 8, 2, 128), ("bf16", 16, 2, 128),
                                            ("f32", 8, 1, 64)])
@pytest.mark.parametrize("top_k,sink,recent,kind", [(1, 0, 1, "random"), (9, 1, 2, "random"),
                                                    (33, 4, 6, "ties"), (64, 0, 1, "random")])
def test_selection_is_exact(pkv, dtype, hq, hkv, d, top_k, sink, recent, kind):
    rng = np.random.default_rng(top_k + hq + d)
    ctx = [1, 16, 17, 1030, 4111, 530, top_k * 16, top_k * 16 + 1]
    case = _select_case(rng, dtype, hq, hkv, d, ctx, [1] * len(ctx), kind)
    t, nb, bounds, exps, q, start = case
    got = _run_select(pkv, dtype, q, bounds, exps, t, ctx, start, top_k, sink, recent,
                      layout=False)
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, start, ctx, 16, top_k, sink, recent, dtype)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 8, 2), ("f32", 4, 4), ("bf16", 8, 1)])
def test_selection_of_several_rows_a_sequence(pkv, dtype, hq, hkv):
    rng = np.random.default_rng(hq + hkv)
    ctx, qlen = [700, 33, 900, 5, 64], [5, 17, 0, 5, 1]
    t, nb, bounds, exps, q, start = _select_case(rng, dtype, hq, hkv, 64, ctx, qlen)
    got = _run_select(pkv, dtype, q, bounds, exps, t, ctx, start, 7, 1, 2, max_ctx=5000, pad=4)
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, start, ctx, 16, 7, 1, 2, dtype)
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("blocks,qlen,hq,top_k", [(20000, 1, 8, 300), (70000, 1, 2, 40),
                                                  (9000, 3, 1, 64), (60000, 2, 1, 1000)])
def test_selection_of_long_contexts(pkv, blocks, qlen, hq, top_k):
    """Keys of tens of thousands of blocks, on chip and (past 49152 of them, or of
    several rows together) through the workspace."""
    rng = np.random.default_rng(blocks)
    ctx = [blocks * 16 - 5, 4097 * 16]
    t, nb, bounds, exps, q, start = _select_case(rng, "bf16", hq, 1, 64, ctx, [qlen, qlen])
    got = _run_select(pkv, "bf16", q, bounds, exps, t, ctx, start, top_k, 1, 2,
                      layout=qlen > 1)
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, start, ctx, 16, top_k, 1, 2, "bf16")
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("kind", ["equal", "near", "spread"])
def test_selection_from_keys_in_few_bins(pkv, kind):
    """Scores that fall into one bin of the key histogram: all equal, a few units
    apart beside an outlier, or spread over the whole range of exponents."""
    rng = np.random.default_rng(3)
    n, d = 3000, 64
    bounds = np.zeros((n, 1, 2, d), np.int8)
    exps = np.zeros((n, 1), np.int8)
    bounds[:, 0, 0, 0] = 64
    if kind == "near":
        bounds[:, 0, 0, 0] = rng.integers(60, 64, n)
        exps[[17, 2000]] = 50
    elif kind == "spread":
        bounds[:, 0, :, 0] = rng.integers(-127, 128, (n, 1))
        exps[:, 0] = rng.integers(-50, 51, n)
    q = np.zeros((1, 1, d), np.float32)
    q[0, 0, 0] = 1.0
    t = rng.permutation(n).astype(np.int32)[None, :]
    for top_k in (3, 4, 700, 2999):
        got = _run_select(pkv, "f32", q, bounds, exps, t, [n * 16], [0, 1], top_k, 1, 1)
        assert pkv.device_error() == 0
        ref = sparse.select(q, bounds, exps, t, [0, 1], [n * 16], 16, top_k, 1, 1, "f32")
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("n", [129, 512, 513, 2048, 2049, 8192, 8193])
@pytest.mark.parametrize("levels", [1, 2, 31, 64, 5000])
def test_selection_at_the_ends_of_the_row_lengths(pkv, n, levels):
    """Rows at the limits of the kernels' lengths, their scores of few or many
    different values, one of them far from the others."""
    rng = np.random.default_rng(n + levels)
    d = 64
    bounds = np.zeros((n, 2, 2, d), np.int8)
    exps = np.zeros((n, 2), np.int8)
    value = rng.integers(0, levels, (n, 2))
    bounds[:, :, 0, 0], bounds[:, :, 0, 1] = value // 100, value % 100
    exps[rng.integers(0, n), 1] = 20
    q = np.zeros((1, 2, d), np.float32)
    q[0, :, 0], q[0, :, 1] = 100.0, 1.0
    t = rng.permutation(n).astype(np.int32)[None, :]
    for top_k, sink, recent in ((2, 0, 1), (5, 1, 2), (100, 4, 30), (n - 1, 1, 1)):
        got = _run_select(pkv, "f32", q, bounds, exps, t, [n * 16], [0, 1], top_k, sink, recent)
        assert pkv.device_error() == 0
        ref = sparse.select(q, bounds, exps, t, [0, 1], [n * 16], 16, top_k, sink, recent, "f32")
        assert np.array_equal(got, ref)


@pytest.mark.parametrize("rows,hq,hkv,qlen", [(41, 16, 8, 1), (23, 32, 8, 2), (14, 8, 8, 3),
                                              (19, 8, 8, 1)])
def test_selection_of_batches_in_long_and_short_stretches(pkv, rows, hq, hkv, qlen):
    """Batches large enough for stretches of 128 or 256 blocks, the last rows in
    shorter ones; contexts of every length among them."""
    rng = np.random.default_rng(rows)
    ctx = [int(x) for x in rng.integers(qlen, 1300 * 16, rows)]
    ctx[0], ctx[-1], ctx[rows // 2] = 1300 * 16, 1299 * 16 + 1, qlen
    lens = [qlen - (i % 3 == 1 and qlen > 1) for i in range(rows)]
    t, nb, bounds, exps, q, start = _select_case(rng, "bf16", hq, hkv, 64, ctx, lens)
    got = _run_select(pkv, "bf16", q, bounds, exps, t, ctx, start, 48, 1, 2, layout=qlen > 1)
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, start, ctx, 16, 48, 1, 2, "bf16")
    assert np.array_equal(got, ref)


def test_selection_with_values_that_are_not_finite(pkv):
    rng = np.random.default_rng(5)
    ctx = [600, 600, 600]
    t, nb, bounds, exps, q, start = _select_case(rng, "f32", 2, 1, 64, ctx, [1, 1, 1])
    exps[t[0, [9, 20]]] = 127                      # blocks that held such a key
    bounds[t[0, [9, 20]]] = 0
    q[1, 0, 3], q[2, :, 7] = np.inf, np.nan        # one head of the group, then both
    got = _run_select(pkv, "f32", q, bounds, exps, t, ctx, start, 5, 1, 1)
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, start, ctx, 16, 5, 1, 1, "f32")
    assert np.array_equal(got, ref)
    assert {9, 20} <= set(got[0, 0].tolist())


def test_zeros_of_either_sign_are_one_score(pkv):
    """A head of negative zeros beside one whose score is 0 or negative: every block
    scores 0, so the lower indices are taken."""
    n, d = 40, 64
    bounds = np.zeros((n, 1, 2, d), np.int8)
    bounds[::2, 0, 0, 0], bounds[::2, 0, 1, 0] = -5, -9
    exps = np.zeros((n, 1), np.int8)
    q = np.full((1, 2, d), -0.0, np.float32)
    q[0, 1, 0] = 1.0
    t = np.arange(n, dtype=np.int32)[None, :]
    for dtype in ("f32", "bf16"):
        qs = q if dtype == "f32" else (q.view(np.uint32) >> 16).astype(np.uint16)
        got = _run_select(pkv, dtype, qs, bounds, exps, t, [n * 16], [0, 1], 8, 0, 1)
        assert got[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, n - 1]
    assert pkv.device_error() == 0


def test_exponents_out_of_range_still_fill_the_list(pkv):
    """Exponents that no bounds call writes order somehow; every entry is a block."""
    rng = np.random.default_rng(21)
    t, nb, bounds, exps, q, start = _select_case(rng, "f32", 2, 1, 64, [800 * 16], [1])
    exps[:, 0] = rng.integers(-128, 128, nb)
    got = _run_select(pkv, "f32", q, bounds, exps, t, [800 * 16], start, 60, 1, 1)
    assert pkv.device_error() == 0
    lst = got[0, 0].tolist()
    assert lst == sorted(set(lst)) and lst[0] == 0 and lst[-1] == 799 and len(lst) == 60


def test_binding_refuses_what_does_not_fit_together(pkv):
    kd = torch.zeros((4, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    desc = pkv.cache_desc(kd, 2)
    bb = pkv.BlockBounds(4, 1, 64)
    t, ctx, start = i32([[0, 1]]), i32([20]), i32([0, 3])
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    sel = torch.full((1, 1, 2), 5, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="num_query_tokens"):
        pkv.pkv_block_bounds(bb.bounds, bb.exps, kd, desc, t, ctx, query_start_loc=start)
    with pytest.raises(ValueError, match="exps: shape"):
        pkv.pkv_block_bounds(bb.bounds, bb.exps[:3].contiguous(), kd, desc, t, ctx)
    with pytest.raises(TypeError, match="k_cache must be a contiguous CUDA"):
        pkv.pkv_block_bounds(bb.bounds, bb.exps, kd.float(), desc, t, ctx)
    with pytest.raises(ValueError, match="block_tables: shape"):
        pkv.pkv_select_blocks(sel, q, bb.bounds, bb.exps, desc, t.t(), ctx, 32, 0, 1)
    with pytest.raises(TypeError, match="block_tables must be a contiguous CUDA"):
        pkv.pkv_select_blocks(sel, q, bb.bounds, bb.exps, desc, i32([[0, 5, 1]])[:, ::2], ctx, 32,
                              0, 1)
    with pytest.raises(ValueError, match="query_start_loc"):
        pkv.paged_attention_sparse(q.repeat(2, 1, 1), q.repeat(2, 1, 1), kd, kd, desc, t, ctx, sel)
    with pytest.raises(ValueError, match="context_lens|block_tables"):
        pkv.paged_attention_sparse(q, q, kd, kd, desc, t, i32([20, 20]), sel,
                                   query_start_loc=i32([0, 1, 1]))
    with pytest.raises(ValueError, match="selected: shape"):
        pkv.paged_attention_sparse(q, q, kd, kd, desc, t, ctx, sel[:, 0])
    with pytest.raises(pkv.PagedKVError):
        pkv.pkv_select_blocks(sel, q, bb.bounds, bb.exps, desc, t, ctx, 32, 2, 1)
    assert (sel == 5).all() and pkv.device_error() == 0


def test_selection_on_a_stream_of_its_own_without_a_workspace(pkv):
    rng = np.random.default_rng(30)
    ctx = [3000, 2000]
    t, nb, bounds, exps, q, start = _select_case(rng, "bf16", 4, 2, 128, ctx, [1, 1])
    desc = pkv.CacheDesc(pkv.PKV_BF16, nb, 16, 2, 4, 128)
    args = [to_dev(q, "bf16"), to_dev(bounds), to_dev(exps), desc, i32(t), i32(ctx)]
    sel = torch.empty((2, 2, 20), dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        pkv.pkv_select_blocks(sel, *args, max(ctx), 1, 1, stream=st)
        torch.full((1 << 16,), 0xFF, dtype=torch.uint8, device="cuda")   # may reuse what is free
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, start, ctx, 16, 20, 1, 1, "bf16")
    assert np.array_equal(sel.cpu().numpy(), ref)


def test_selection_flags_bad_batches(pkv):
    rng = np.random.default_rng(6)
    ctx = [600, 90, 300]
    t, nb, bounds, exps, q, start = _select_case(rng, "bf16", 2, 1, 64, ctx, [1, 1, 1])
    bad = t.copy()
    bad[0, 5], bad[0, 6] = -1, nb
    got = _run_select(pkv, "bf16", q, bounds, exps, bad, ctx, start, 4, 1, 1)
    assert pkv.device_error() == 1
    assert np.array_equal(got, sparse.select(q, bounds, exps, bad, start, ctx, 16, 4, 1, 1,
                                             "bf16"))
    for c, code in (([600, 0, 300], 2), ([600, 700, 300], 2), ([600, -3, 300], 2)):
        got = _run_select(pkv, "bf16", q, bounds, exps, t, c, start, 4, 1, 1, max_ctx=640)
        assert pkv.device_error() == code
        ok = sparse.select(q, bounds, exps, t, start, ctx, 16, 4, 1, 1, "bf16")
        assert (got[1] == -1).all() and np.array_equal(got[[0, 2]], ok[[0, 2]])
    got = _run_select(pkv, "bf16", q, bounds, exps, t[:, :20].copy(), ctx, start, 4, 1, 1)
    assert pkv.device_error() == 7 and (got[0] == -1).all()


# ---- attention -----------------------------------------------------------------
def _lists(rng, ctx, start, hkv, top_k, kind="sorted"):
    rows = int(start[-1])
    sel = np.full((rows, hkv, top_k), -1, dtype=np.int32)
    for r, s, keys in sparse.row_layout(start, ctx):
        n = -(-keys // 16)
        for h in range(hkv):
            pick = rng.permutation(n)[:top_k]
            if kind == "sorted":
                pick = np.sort(pick)
            elif kind == "holes":                  # skipped entries between, order as it comes
                pick = np.where(rng.random(len(pick)) < 0.3, -1 - pick, pick)
            elif kind == "twice":
                pick = np.concatenate([pick, pick])[:top_k]
            sel[r, h, :len(pick)] = pick
    return sel


def _run_attend(pkv, dtype, q, k, v, t, ctx, start, sel, pad=0, layout=True, scale=None):
    kd, vd = to_dev(k, dtype), to_dev(v, dtype)
    qp = np.concatenate([q, np.zeros((pad,) + q.shape[1:], q.dtype)])
    qd = to_dev(qp, dtype)
    out = torch.full_like(qd, 7.0)
    selp = np.concatenate([sel, np.zeros((pad,) + sel.shape[1:], sel.dtype)])
    pkv.paged_attention_sparse(out, qd, kd, vd, pkv.cache_desc(kd, q.shape[1]), i32(t), i32(ctx),
                               i32(selp), query_start_loc=i32(start) if layout else None,
                               scale=scale)
    assert (out[q.shape[0]:] == 7.0).all()
    return out[:q.shape[0]]


def _attend_case(rng, dtype, hq, hkv, d, ctx, qlen, top_k, kind="sorted", scale=1.0):
    start = np.concatenate([[0], np.cumsum(qlen)])
    t, nb = tables_for(rng, ctx)
    k, v = (_poison(values(rng, (nb, hkv, 16, d), dtype, scale), t, ctx, dtype) for _ in range(2))
    q = values(rng, (int(start[-1]), hq, d), dtype, scale)
    return q, k, v, t, start, _lists(rng, ctx, start, hkv, top_k, kind)


def _check_attend(pkv, dtype, q, k, v, t, ctx, start, sel, scale=None, **kw):
    out = _run_attend(pkv, dtype, q, k, v, t, ctx, start, sel, scale=scale, **kw)
    assert pkv.device_error() == 0
    ref = sparse.attention(q, k, v, t, start, ctx, sel, dtype, scale)
    assert_attention(out, ref, attention_bound(q, k, v, t, start, ctx, sel, dtype, ref, scale))


GROUPS = [(8, 8), (8, 4), (8, 2), (16, 2), (5, 5), (8, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", GROUPS)
def test_attention_over_lists(pkv, dtype, d, hq, hkv):
    rng = np.random.default_rng(hq * 10 + hkv + d)
    ctx = [1, 16, 17, 1030, 530, 95]
    q, k, v, t, start, sel = _attend_case(rng, dtype, hq, hkv, d, ctx, [1] * 6, 21)
    _check_attend(pkv, dtype, q, k, v, t, ctx, start, sel, layout=False)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 1, 128), ("bf16", 4, 4, 64),
                                            ("f32", 4, 2, 128)])
@pytest.mark.parametrize("kind,top_k", [("sorted", 1), ("holes", 13), ("twice", 40),
                                        ("sorted", 200)])
def test_attention_of_several_rows_a_sequence(pkv, dtype, hq, hkv, d, kind, top_k):
    rng = np.random.default_rng(top_k + hq)
    ctx, qlen = [700, 33, 900, 5, 64, 2000], [5, 17, 0, 5, 1, 2]
    q, k, v, t, start, sel = _attend_case(rng, dtype, hq, hkv, d, ctx, qlen, top_k, kind)
    _check_attend(pkv, dtype, q, k, v, t, ctx, start, sel, pad=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 40])
def test_attention_over_long_lists_of_few_and_many_rows(pkv, dtype, rows):
    """Lists longer than a warp's prefetch of 32 tiles, shared by one CTA or a cluster."""
    rng = np.random.default_rng(rows)
    ctx = [int(x) for x in rng.integers(6000, 9000, rows)]
    q, k, v, t, start, sel = _attend_case(rng, dtype, 4, 1, 128, ctx, [1] * rows, 513)
    _check_attend(pkv, dtype, q, k, v, t, ctx, start, sel)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_attention_with_large_scores_and_other_scales(pkv, dtype, d):
    rng = np.random.default_rng(d)
    ctx = [900, 350, 40]
    case = _attend_case(rng, dtype, 8, 2, d, ctx, [1, 1, 1], 30, scale=4.0)
    q, k, v, t, start, sel = case
    for scale in (None, 0.7, -0.2, 0.0):
        _check_attend(pkv, dtype, q, k, v, t, ctx, start, sel, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lists_that_leave_a_row_empty_give_zeros(pkv, dtype):
    rng = np.random.default_rng(2)
    ctx = [300, 20]
    q, k, v, t, start, sel = _attend_case(rng, dtype, 4, 2, 128, ctx, [1, 1], 6)
    sel[0, 1] = -1
    sel[1, 0] = -5
    out = _run_attend(pkv, dtype, q, k, v, t, ctx, start, sel)
    assert pkv.device_error() == 0
    assert (out[0, 2:] == 0).all() and (out[1, :2] == 0).all()
    ref = sparse.attention(q, k, v, t, start, ctx, sel, dtype)
    assert_attention(out, ref, attention_bound(q, k, v, t, start, ctx, sel, dtype, ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_of_minus_infinity(pkv, dtype):
    """A whole block of keys whose scores are -inf weighs nothing; a NaN key shows."""
    rng = np.random.default_rng(9)
    ctx = [200, 200]
    q, k, v, t, start, sel = _attend_case(rng, dtype, 2, 1, 64, ctx, [1, 1], 13)
    one, inf, nan = ((1.0, -np.inf, np.nan) if dtype == "f32"
                     else (np.uint16(0x3F80), np.uint16(0xFF80), NAN_BITS))
    q[0, :, 0] = one
    k[t[0, 0], 0, :, 0] = inf                     # the first listed block
    k[t[1, 3], 0, 4, 0] = nan
    out = _run_attend(pkv, dtype, q, k, v, t, ctx, start, sel)
    assert pkv.device_error() == 0
    assert torch.isnan(out[1]).all()
    with np.errstate(invalid="ignore"):
        ref = sparse.attention(q, k, v, t, start, ctx, sel, dtype)
    bare = sel.copy()
    bare[0, 0][bare[0, 0] == 0] = -1
    ref0 = sparse.attention(q[:1], k, v, t[:1], [0, 1], ctx[:1], bare[:1], dtype)
    assert np.abs(ref[0] - ref0[0]).max() < 1e-12
    bound = attention_bound(q[:1], k, v, t[:1], [0, 1], ctx[:1], bare[:1], dtype, ref0)
    assert_attention(out[:1], ref0, bound)


@pytest.mark.parametrize("top_k", [3, 40])
@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("bf16", 4, 4, 64),
                                            ("f32", 4, 2, 64)])
def test_infinite_values_stay_infinite(pkv, dtype, hq, hkv, d, top_k):
    """A visible value of +-inf makes its element infinite and no other (each
    weight is above 2^-100: scores lie within 30 of one another)."""
    rng = np.random.default_rng(29)
    n = top_k * 16 - 5
    t, nb = tables_for(rng, [n])
    k, v = (values(rng, (nb, hkv, 16, d), dtype) for _ in range(2))
    q = values(rng, (1, hq, d), dtype, 0.5)
    vt = to_dev(v, dtype)
    for at, dim, x in ((0, 3, float("inf")), (n - 1, 3, float("inf")), (n // 2, 8, -float("inf"))):
        vt[int(t[0, at // 16]), :, at % 16, dim] = x
    desc = pkv.CacheDesc({"bf16": pkv.PKV_BF16, "f32": pkv.PKV_F32}[dtype], nb, 16, hkv, hq, d)
    sel = i32(np.tile(np.arange(top_k), (1, hkv, 1)))
    qt, kt = to_dev(q, dtype), to_dev(k, dtype)
    out, clean = torch.empty_like(qt), torch.empty_like(qt)
    pkv.paged_attention_sparse(out, qt, kt, vt, desc, i32(t), i32([n]), sel)
    pkv.paged_attention_sparse(clean, qt, kt, to_dev(v, dtype), desc, i32(t), i32([n]), sel)
    assert pkv.device_error() == 0
    clean[:, :, 3], clean[:, :, 8] = float("inf"), -float("inf")
    assert torch.equal(out, clean)


def test_attention_flags_bad_entries(pkv):
    rng = np.random.default_rng(4)
    ctx = [300, 20]
    q, k, v, t, start, sel = _attend_case(rng, "bf16", 4, 2, 128, ctx, [1, 1], 6)
    ref = sparse.attention(q, k, v, t, start, ctx, sel, "bf16")
    bound = attention_bound(q, k, v, t, start, ctx, sel, "bf16", ref)
    bad = sel.copy()
    bad[1, :, 3] = 2                               # past the row's two blocks
    out = _run_attend(pkv, "bf16", q, k, v, t, ctx, start, bad)
    assert pkv.device_error() == 1
    assert_attention(out, ref, bound)
    tb = t.copy()
    tb[0, 0] = k.shape[0]                          # outside the pool
    drop = sel.copy()
    drop[0][drop[0] == 0] = -1
    out = _run_attend(pkv, "bf16", q, k, v, tb, ctx, start, sel)
    assert pkv.device_error() == 1
    refd = sparse.attention(q, k, v, t, start, ctx, drop, "bf16")
    assert_attention(out, refd, attention_bound(q, k, v, t, start, ctx, drop, "bf16", refd))
    out = _run_attend(pkv, "bf16", q, k, v, t, [300, 0], start, sel)
    assert pkv.device_error() == 2 and (out[1] == 0).all()


@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 16, 8), ("bf16", 8, 8)])
def test_tiles_past_32_bits_of_the_pool(pkv, dtype, hq, hkv):
    """A pool of more than 2^31 elements, and 2^32 bytes: blocks at its end."""
    nb, d = 140000, 128
    rng = np.random.default_rng(1)
    kd = torch.empty((nb, hkv, 16, d), dtype=torch.bfloat16, device="cuda")
    vd = torch.empty_like(kd)
    assert kd.numel() > 1 << 31
    n = 24
    k, v = (values(rng, (n, hkv, 16, d), dtype) for _ in range(2))
    ids = nb - n + np.arange(n)
    kd[nb - n:], vd[nb - n:] = to_dev(k, dtype), to_dev(v, dtype)
    q = values(rng, (1, hq, d), dtype)
    ctx, start = [n * 16 - 3], [0, 1]
    local = rng.permutation(n).astype(np.int32)[None, :]
    sel = _lists(rng, ctx, start, hkv, 20)
    out = torch.empty((1, hq, d), dtype=torch.bfloat16, device="cuda")
    pkv.paged_attention_sparse(out, to_dev(q, dtype), kd, vd, pkv.cache_desc(kd, hq),
                               i32(ids[local]), i32(ctx), i32(sel))
    bounds = torch.zeros((nb, hkv, 2, d), dtype=torch.int8, device="cuda")
    exps = torch.zeros((nb, hkv), dtype=torch.int8, device="cuda")
    pkv.pkv_block_bounds(bounds, exps, kd, pkv.cache_desc(kd, hq), i32(ids[local]), i32(ctx),
                         query_start_loc=i32([0, ctx[0]]), num_query_tokens=ctx[0])
    assert pkv.device_error() == 0
    ref = sparse.attention(q, k, v, local, start, ctx, sel, dtype)
    assert_attention(out, ref, attention_bound(q, k, v, local, start, ctx, sel, dtype, ref))
    b, e = np.zeros((n, hkv, 2, d), np.int8), np.zeros((n, hkv), np.int8)
    sparse.update_bounds(b, e, k, local, [0, ctx[0]], ctx, dtype)
    assert np.array_equal(bounds[nb - n:].cpu().numpy(), b)
    assert np.array_equal(exps[nb - n:].cpu().numpy(), e)


def test_bounds_past_32_bits_of_their_pool(pkv):
    """More than 2^31 bytes of bounds: blocks at the end of the pool are scored."""
    nb, hkv, d, n = 1 << 20, 9, 128, 300
    bd = torch.empty((nb, hkv, 2, d), dtype=torch.int8, device="cuda")
    ed = torch.empty((nb, hkv), dtype=torch.int8, device="cuda")
    assert bd.numel() > 1 << 31
    rng = np.random.default_rng(19)
    t, _, bounds, exps, q, start = _select_case(rng, "bf16", 2 * hkv, hkv, d, [n * 16], [1])
    ids = nb - bounds.shape[0] + np.arange(bounds.shape[0])
    bd[nb - bounds.shape[0]:], ed[nb - bounds.shape[0]:] = to_dev(bounds), to_dev(exps)
    desc = pkv.CacheDesc(pkv.PKV_BF16, nb, 16, hkv, 2 * hkv, d)
    sel = torch.empty((1, hkv, 40), dtype=torch.int32, device="cuda")
    pkv.pkv_select_blocks(sel, to_dev(q, "bf16"), bd, ed, desc, i32(ids[t]), i32([n * 16]), n * 16,
                          1, 1)
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, start, [n * 16], 16, 40, 1, 1, "bf16")
    assert np.array_equal(sel.cpu().numpy(), ref)


def test_two_captured_selections_share_a_workspace(pkv):
    """Two graphs with one workspace, replayed in turn: nothing stays in it."""
    rng = np.random.default_rng(23)
    calls = []
    ws = pkv.workspace(8 << 20)
    for ctx in ([2500, 900, 40], [700, 4000]):
        t, nb, bounds, exps, q, start = _select_case(rng, "bf16", 8, 2, 64, ctx, [1] * len(ctx))
        desc = pkv.CacheDesc(pkv.PKV_BF16, nb, 16, 2, 8, 64)
        args = (to_dev(q, "bf16"), to_dev(bounds), to_dev(exps), desc, i32(t), i32(ctx), max(ctx))
        sel = torch.full((len(ctx), 2, 30), -9, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pkv.pkv_select_blocks(sel, *args, 1, 1, ws=ws)
        ref = sparse.select(q, bounds, exps, t, start, ctx, 16, 30, 1, 1, "bf16")
        calls.append((g, sel, ref, args))
    for _ in range(4):
        for g, sel, ref, _ in calls:
            sel.fill_(-9)
            g.replay()
            assert np.array_equal(sel.cpu().numpy(), ref)
    assert pkv.device_error() == 0


# ---- together ------------------------------------------------------------------
class Serving:
    """A batch served from the device: tables, append, bounds, selection and sparse
    attention of each step enqueued one behind the other, nothing read back."""

    def __init__(self, pkv, dtype, n, hq, hkv, d, top_k, blocks_each=40):
        self.pkv, self.n, self.top_k = pkv, n, top_k
        tdt = torch.float32 if dtype == "f32" else torch.bfloat16
        nb = n * blocks_each
        self.kc = torch.full((nb, hkv, 16, d), float("nan"), dtype=tdt, device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        self.desc = pkv.cache_desc(self.kc, hq)
        self.bb = pkv.BlockBounds(nb, hkv, d)
        self.order = np.random.default_rng(n).permutation(nb)
        self.dt = pkv.DeviceTables.create(nb, 16, n + 3, blocks_each, self.order)
        self.rows = i32(np.random.default_rng(7).permutation(n + 3)[:n])
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.tables = torch.empty((n, blocks_each), dtype=torch.int32, device="cuda")
        self.max_ctx = blocks_each * 16

    def buffers(self, tokens):
        hkv, d, hq = self.desc.num_kv_heads, self.desc.head_dim, self.desc.num_q_heads
        self.start = torch.empty(self.n + 1, dtype=torch.int32, device="cuda")
        self.slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
        self.sel = torch.empty((tokens, hkv, self.top_k), dtype=torch.int32, device="cuda")
        self.out = torch.empty((tokens, hq, d), dtype=self.kc.dtype, device="cuda")
        self.ws = self.pkv.workspace(self.pkv.select_workspace_bytes(self.desc, tokens,
                                                                     self.max_ctx))

    def step(self, q, k, v, new=None):
        p = self.pkv
        p.pkv_tables_step(self.dt, self.rows, self.lens, new, self.tables, self.lens, self.start,
                          self.slots)
        p.paged_kv_append(k, v, self.slots, self.kc, self.vc, self.desc)
        p.pkv_block_bounds(self.bb.bounds, self.bb.exps, self.kc, self.desc, self.tables,
                           self.lens, query_start_loc=self.start, num_query_tokens=q.shape[0])
        p.pkv_select_blocks(self.sel, q, self.bb.bounds, self.bb.exps, self.desc, self.tables,
                            self.lens, self.max_ctx, 1, 2, query_start_loc=self.start, ws=self.ws)
        p.paged_attention_sparse(self.out, q, self.kc, self.vc, self.desc, self.tables, self.lens,
                                 self.sel, query_start_loc=self.start)


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("f32", 4, 4, 64)])
def test_prompts_then_captured_decode_steps(pkv, dtype, hq, hkv, d):
    n, top_k, steps = 5, 12, 20
    rng = np.random.default_rng(hq)
    sv = Serving(pkv, dtype, n, hq, hkv, d, top_k)
    prompts = [300, 17, 1, 555, 160]
    tokens = sum(prompts) + 6                      # padded
    # prompts: every prompt row selects and attends too
    sv.buffers(tokens)
    q, k, v = (values(rng, (tokens, h, d), dtype) for h in (hq, hkv, hkv))
    sv.out.fill_(7.0)
    sv.step(to_dev(q, dtype), to_dev(k, dtype), to_dev(v, dtype), i32(prompts))
    assert pkv.device_error() == 0
    model = sparse.TablesModel(sv.kc.shape[0], 16, n + 3, 40, sv.order)
    rows = sv.rows.cpu().tolist()
    ok, ov = np.zeros(tuple(sv.kc.shape), k.dtype), np.zeros(tuple(sv.kc.shape), k.dtype)
    bounds = np.zeros(tuple(sv.bb.bounds.shape), np.int8)
    exps = np.zeros(tuple(sv.bb.exps.shape), np.int8)

    def check(q, k, v, cached, new):
        ctx, start, slots, _, tables = model.step(rows, cached, new, q.shape[0], 40)
        live = slots >= 0
        ocache.append(ok, ov, k[live], v[live], slots[live], 16)
        sparse.update_bounds(bounds, exps, ok, tables, start, ctx, dtype)
        ref_sel = sparse.select(q, bounds, exps, tables, start, ctx, 16, top_k, 1, 2, dtype)
        assert np.array_equal(sv.tables.cpu().numpy(), tables)
        assert np.array_equal(sv.bb.bounds.cpu().numpy(), bounds)
        m = int(start[-1])
        assert np.array_equal(sv.sel.cpu().numpy()[:m], ref_sel[:m])
        ref = sparse.attention(q[:m], ok, ov, tables, start, ctx, ref_sel, dtype)
        assert_attention(sv.out[:m], ref, attention_bound(q[:m], ok, ov, tables, start, ctx,
                                                          ref_sel, dtype, ref))
        return ctx

    lens = check(q, k, v, [0] * n, prompts)
    assert (sv.out[sum(prompts):] == 7.0).all()
    # decode: one captured step, replayed over inputs copied in place
    sv.buffers(n)
    qd, kd, vd = (torch.zeros((n, h, d), dtype=sv.kc.dtype, device="cuda") for h in (hq, hkv, hkv))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        sv.step(qd, kd, vd)
    for _ in range(steps):
        q, k, v = (values(rng, (n, h, d), dtype) for h in (hq, hkv, hkv))
        qd.copy_(to_dev(q, dtype))
        kd.copy_(to_dev(k, dtype))
        vd.copy_(to_dev(v, dtype))
        g.replay()
        lens = check(q, k, v, lens, None)
    assert pkv.device_error() == 0
    assert sv.lens.tolist() == [p + steps for p in prompts]


def test_all_blocks_selected_is_dense_decode(pkv):
    rng = np.random.default_rng(12)
    ctx = [900, 77, 16, 333]
    t, nb = tables_for(rng, ctx)
    k, v = (values(rng, (nb, 2, 16, 128), "bf16", 0.5) for _ in range(2))
    q = values(rng, (4, 8, 128), "bf16", 0.5)
    kd, vd, qd = (to_dev(x, "bf16") for x in (k, v, q))
    desc = pkv.cache_desc(kd, 8)
    bb = pkv.BlockBounds(nb, 2, 128)
    start = i32(np.concatenate([[0], np.cumsum(ctx)]))
    pkv.pkv_block_bounds(bb.bounds, bb.exps, kd, desc, i32(t), i32(ctx), query_start_loc=start,
                         num_query_tokens=sum(ctx))
    sel = torch.empty((4, 2, 60), dtype=torch.int32, device="cuda")
    pkv.pkv_select_blocks(sel, qd, bb.bounds, bb.exps, desc, i32(t), i32(ctx), 900, 0, 1)
    out = pkv.paged_attention_sparse(torch.empty_like(qd), qd, kd, vd, desc, i32(t), i32(ctx),
                                     sel)
    assert pkv.device_error() == 0
    ref = oatt.decode(q, k, v, t, ctx, 16, "bf16")
    assert_attention(out, ref, attention_bound(q, k, v, t, np.arange(5), ctx,
                                               sel.cpu().numpy(), "bf16", ref))


def test_calls_on_two_streams_do_not_disturb_each_other(pkv):
    """Two batches on two streams at once, each with a workspace of its own."""
    rng = np.random.default_rng(15)
    got, want = [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        ctx = [int(x) for x in rng.integers(500, 3000, 6)]
        t, nb, bounds, exps, q, start = _select_case(rng, "bf16", 8, 2, 128, ctx, [1] * 6)
        k, v = (values(rng, (nb, 2, 16, 128), "bf16") for _ in range(2))
        kd, vd, qd, bd, ed = (to_dev(k, "bf16"), to_dev(v, "bf16"), to_dev(q, "bf16"),
                              to_dev(bounds), to_dev(exps))
        td, cd = i32(t), i32(ctx)
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            desc = pkv.cache_desc(kd, 8)
            sel = torch.empty((6, 2, 20), dtype=torch.int32, device="cuda")
            out = torch.empty_like(qd)
            for _ in range(20):
                pkv.pkv_select_blocks(sel, qd, bd, ed, desc, td, cd, max(ctx), 1, 1)
                pkv.paged_attention_sparse(out, qd, kd, vd, desc, td, cd, sel)
        got.append((sel, out, (kd, vd, bd, ed, td, cd)))
        want.append((q, k, v, t, start, ctx, bounds, exps))
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    for (sel, out, _), (q, k, v, t, start, ctx, bounds, exps) in zip(got, want):
        ref_sel = sparse.select(q, bounds, exps, t, start, ctx, 16, 20, 1, 1, "bf16")
        assert np.array_equal(sel.cpu().numpy(), ref_sel)
        ref = sparse.attention(q, k, v, t, start, ctx, ref_sel, "bf16")
        assert_attention(out, ref, attention_bound(q, k, v, t, start, ctx, ref_sel, "bf16", ref))
