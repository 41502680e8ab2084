"""GPU: latent attention over a paged cache (append, copies, gather, absorbed attention)
against the float64 restatement."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import latent, rope  # noqa: E402
from oracle.numerics import widen  # noqa: E402
from tests.gpu_parity import gamma  # noqa: E402
from tests.latent_checks import absorbed_bound, assert_close, fill, latent_cache  # noqa: E402
from tests.sparse_checks import ROUND, i32, tables_for, to_dev, values  # noqa: E402
from tests.test_gpu_sparse_layouts import fenced  # noqa: E402

pytestmark = pytest.mark.gpu

SCALE = 192.0 ** -0.5


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


def host(t):
    t = t.cpu()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


# ------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r,h,interleaved,normed", [(128, 1, True, True), (256, 17, False, True),
                                                    (384, 32, True, False), (512, 5, False, False),
                                                    (512, 48, True, True)])
@pytest.mark.parametrize("tokens", [1, 7, 700])
def test_append(pkv, dtype, r, h, interleaved, normed, tokens):
    """Rows land in their slots; copies and rotations bit for bit; the norm within its
    roundings: gamma_{r + 8} of a sum of r squares, its root, three products, then half a
    step of the type.  Inputs and q_out are parts of wider tensors."""
    rng = np.random.default_rng(r + h + tokens)
    nb = -(-tokens // 16) + 3
    down = values(rng, (tokens, r + 64), dtype, 3.0)
    q = values(rng, (tokens, h, 96 + 64), dtype)
    w = values(rng, (r,), dtype) if normed else None
    slots = rng.permutation(nb * 16)[:tokens].astype(np.int64)
    slots[2::5] = -1
    pos = rng.integers(0, 300, tokens).astype(np.int32)
    tab = rope.rope_table(300, 64)
    a, b, done = latent.append(down[:, :r], np.ascontiguousarray(down[:, r:]), slots, pos, tab, 16,
                               nb, dtype, w, 1e-5, interleaved)
    cos, sin = latent.angles(tab, pos)
    q_ref = latent.rotate(np.ascontiguousarray(q[..., 96:]), cos[:, None], sin[:, None],
                          interleaved, dtype)
    dd, qd = to_dev(down, dtype), to_dev(q, dtype)
    cache, whole = fenced(to_dev(latent_cache(rng, nb, r, dtype, 0), dtype))
    wide = torch.full((tokens, h, r + 64), 7.0, dtype=qd.dtype, device="cuda")
    desc = pkv.latent_desc(cache, r, h)
    pkv.paged_latent_append(dd[:, :r], dd[:, r:], torch.from_numpy(slots).cuda(), i32(pos),
                            to_dev(tab), cache, desc, None if w is None else to_dev(w, dtype),
                            1e-5, qd[..., 96:], wide[..., r:], interleaved)
    assert pkv.device_error() == 0 and whole()
    got = host(cache)
    assert np.array_equal(got[..., r:][done], b[done])
    assert (got[~done] == 0).all()
    if normed:
        bound = (gamma(r + 8) + ROUND[dtype]) * np.abs(a) + 1e-30
        assert (np.abs(widen(got[..., :r], dtype) - a)[done] <= bound[done]).all()
    else:
        assert np.array_equal(widen(got[..., :r], dtype)[done], a[done])
    assert np.array_equal(host(wide[..., r:].contiguous()), q_ref)
    assert (wide[..., :r] == 7.0).all()
    # in place, and without queries
    pkv.paged_latent_append(dd[:, :r], dd[:, r:], torch.from_numpy(slots).cuda(), i32(pos),
                            to_dev(tab), cache, desc, q=qd[..., 96:], interleaved=interleaved)
    assert np.array_equal(host(qd[..., 96:].contiguous()), q_ref)
    assert np.array_equal(host(qd[..., :96].contiguous()), q[..., :96])
    pkv.paged_latent_append(dd[:, :r], dd[:, r:], torch.from_numpy(slots).cuda(), i32(pos),
                            to_dev(tab), cache, desc, interleaved=interleaved)
    assert pkv.device_error() == 0 and whole()
    assert np.array_equal(host(cache)[..., :r][done], down[:, :r][_order(slots, done)])


def _order(slots, done):
    """Tokens in the order in which `done` lists their slots."""
    where = {int(s): t for t, s in enumerate(slots) if s >= 0}
    return [where[int(s)] for s in np.flatnonzero(done.reshape(-1))]


@pytest.mark.parametrize("bad,code", [("slot", 3), ("position", 8), ("negative", 8)])
def test_append_skips_and_flags(pkv, bad, code):
    cache = torch.zeros((2, 16, 192), device="cuda")
    desc = pkv.latent_desc(cache, 128, 2)
    x, k, q = torch.ones(2, 128).cuda(), torch.ones(2, 64).cuda(), torch.ones(2, 2, 64).cuda()
    slots = torch.tensor([32 if bad == "slot" else 5, 6]).cuda()
    pos = i32([8 if bad == "position" else -1 if bad == "negative" else 1, 1])
    out = torch.full_like(q, 9.0)
    pkv.paged_latent_append(x, k, slots, pos, to_dev(rope.rope_table(8, 64)), cache, desc, q=q,
                            q_out=out)
    assert pkv.device_error() == code
    assert (cache[0, 6, :128] == 1).all() and int((cache != 0).any(-1).sum()) == 1
    assert bool((out[0] == 9.0).all()) == (bad != "slot") and (out[1] != 9.0).any()


def test_copy_blocks(pkv):
    rng = np.random.default_rng(3)
    for dtype in ("bf16", "f32"):
        c = values(rng, (9, 16, 320), dtype)
        cd = to_dev(c, dtype)
        desc = pkv.latent_desc(cd, 256, 4)
        pkv.pkv_copy_blocks_latent(i32([[0, 8], [3, 1]]), cd, desc)
        assert pkv.device_error() == 0
        want = c.copy()
        want[8], want[1] = c[0], c[3]
        assert np.array_equal(host(cd), want)
        pkv.pkv_copy_blocks_latent(i32([[0, 9], [2, 7]]), cd, desc)
        assert pkv.device_error() == 4
        want[7] = want[2]
        assert np.array_equal(host(cd), want)


# ------------------------------------------------------------------------------------
# gather
# ------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r", [128, 256, 384, 512])
@pytest.mark.parametrize("lens", [[1], [16, 17, 15], [0, 3, 0, 0, 130, 1], [1] * 70 + [33]])
def test_gather(pkv, dtype, r, lens):
    """Rows bit for bit; rows behind the last sequence, and what surrounds the outputs, as
    they were."""
    rng = np.random.default_rng(sum(lens) + r)
    t, nb = tables_for(rng, [max(n, 1) for n in lens])
    c = values(rng, (nb, 16, r + 64), dtype)
    starts, n = np.concatenate([[0], np.cumsum(lens)]), sum(lens)
    cd = to_dev(c, dtype)
    x, x_whole = fenced(torch.full((n + 5, r), 3.0, dtype=cd.dtype, device="cuda"))
    k, k_whole = fenced(torch.full((n + 5, 64), 3.0, dtype=cd.dtype, device="cuda"))
    pkv.paged_latent_gather(x, k, cd, pkv.latent_desc(cd, r, 1), i32(t), i32(starts))
    assert pkv.device_error() == 0 and x_whole() and k_whole()
    want = np.concatenate([latent.rows_of(c, t[s], m) for s, m in enumerate(lens)])
    assert np.array_equal(host(x)[:n], want[:, :r]) and np.array_equal(host(k)[:n], want[:, r:])
    assert (x[n:] == 3.0).all() and (k[n:] == 3.0).all()


@pytest.mark.parametrize("fault,code", [("id", 1), ("minus", 1), ("narrow", 7), ("falls", 5),
                                        ("late", 5), ("above", 5)])
def test_gather_leaves_rows_that_it_cannot_read(pkv, fault, code):
    rng = np.random.default_rng(9)
    t, nb = tables_for(rng, [40, 40])
    c = values(rng, (nb, 16, 192), "f32")
    starts, n = [0, 40, 80], 80
    if fault in ("id", "minus"):
        t[1, 1] = nb if fault == "id" else -3
    if fault == "narrow":
        t = t[:, :2]
    if fault == "falls":
        starts = [0, 60, 50]
    if fault == "late":
        starts = [3, 40, 80]
    if fault == "above":
        starts = [0, 40, 81]
    cd = to_dev(c)
    x, x_whole = fenced(torch.full((n, 128), 3.0, device="cuda"))
    k, k_whole = fenced(torch.full((n, 64), 3.0, device="cuda"))
    pkv.paged_latent_gather(x, k, cd, pkv.latent_desc(cd, 128, 1), i32(t), i32(starts))
    assert pkv.device_error() == code and x_whole() and k_whole()
    kept = (host(x) == 3.0).all(1)
    left = {"id": range(56, 72), "minus": range(56, 72), "above": range(80), "late": range(3),
            "narrow": [*range(32, 40), *range(72, 80)]}
    if fault in left:
        assert sorted(np.flatnonzero(kept)) == list(left[fault])


# ------------------------------------------------------------------------------------
# absorbed attention
# ------------------------------------------------------------------------------------
def attend(pkv, q, cache, t, ctx, dtype, start=None, most=None, scale=SCALE, ws_byte=0xFF, **kw):
    """(output, device error): outputs and workspace between fences, the workspace full of
    NaN beforehand."""
    qd, cd = to_dev(q, dtype), to_dev(cache, dtype)
    r = cache.shape[2] - 64
    desc = pkv.latent_desc(cd, r, q.shape[1])
    out, out_whole = fenced(torch.full(q.shape[:2] + (r,), 7.0, dtype=cd.dtype, device="cuda"))
    need = pkv.latent_workspace_bytes(desc, len(ctx), q.shape[0], most or max(ctx))
    ws, ws_whole = fenced(torch.full((need,), ws_byte, dtype=torch.uint8, device="cuda"))
    pkv.paged_attention_latent(out, qd, cd, desc, i32(t), i32(ctx), most or max(ctx), scale,
                               None if start is None else i32(start), ws, **kw)
    code = pkv.device_error()
    assert out_whole() and ws_whole()
    return out, code


def batch(rng, dtype, r, ctx, hidden=True):
    """(pool, tables): every sequence's rows random, all other rows NaN."""
    t, nb = tables_for(rng, ctx)
    cache = latent_cache(rng, nb, r, dtype)
    for s, n in enumerate(ctx):
        fill(cache, t[s], values(rng, (n, r + 64), dtype))
    return cache, t


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r", [128, 256, 384, 512])
@pytest.mark.parametrize("h", [1, 3, 8, 24, 64])
def test_one_token_a_sequence(pkv, dtype, r, h):
    """Contexts around block and tile edges, in no order; rows of the pool that no token
    was written to hold NaN."""
    ctx = [1, 16, 33, 2, 15, 17, 31, 32, 64, 65, 63, 200]
    rng = np.random.default_rng(r + h)
    cache, t = batch(rng, dtype, r, ctx)
    q = values(rng, (len(ctx), h, r + 64), dtype)
    start = np.arange(len(ctx) + 1)
    ref = latent.absorbed(q, cache, t, start, ctx, SCALE, dtype)
    out, code = attend(pkv, q, cache, t, ctx, dtype)
    assert code == 0
    assert_close(out, ref, absorbed_bound(q, cache, t, start, ctx, SCALE, dtype, ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r,h,new,ctx", [
    (128, 5, [3, 0, 1, 7, 2], [3, 9, 1, 100, 50]),
    (512, 24, [3, 3, 3], [40, 130, 3]),
    (256, 128, [2, 1], [70, 33]),
    (384, 2, [40, 64], [40, 500]),
    (512, 65, [1, 1, 1], [5, 500, 64]),
    (128, 40, [33], [300]),
])
def test_several_tokens_a_sequence(pkv, dtype, r, h, new, ctx):
    """Row i sees keys 0 .. ctx - qlen + i; sequences without queries, prompts that are
    their own context, more rows than a team of CTAs takes."""
    rng = np.random.default_rng(h)
    cache, t = batch(rng, dtype, r, ctx)
    start = np.concatenate([[0], np.cumsum(new)])
    q = values(rng, (start[-1] + 3, h, r + 64), dtype)        # three rows of padding
    ref = latent.absorbed(q, cache, t, start, ctx, SCALE, dtype)
    out, code = attend(pkv, q, cache, t, ctx, dtype, start)
    assert code == 0
    assert_close(out, ref, absorbed_bound(q, cache, t, start, ctx, SCALE, dtype, ref))
    assert (out[start[-1]:] == 7.0).all()


@pytest.mark.parametrize("dtype,r,h,ctx", [("bf16", 512, 16, [9000, 40, 3]),
                                           ("bf16", 128, 100, [5000]),
                                           ("f32", 256, 8, [6000, 1]),
                                           ("bf16", 256, 4, [30] * 400),
                                           ("f32", 128, 2, [20] * 400)])
def test_long_contexts_and_many_sequences(pkv, dtype, r, h, ctx):
    """Units cut over many CTAs and joined; more sequences than a CTA has threads."""
    rng = np.random.default_rng(len(ctx))
    cache, t = batch(rng, dtype, r, ctx)
    q = values(rng, (len(ctx), h, r + 64), dtype)
    start = np.arange(len(ctx) + 1)
    ref = latent.absorbed(q, cache, t, start, ctx, SCALE, dtype)
    bound = absorbed_bound(q, cache, t, start, ctx, SCALE, dtype, ref)
    out, code = attend(pkv, q, cache, t, ctx, dtype)
    assert code == 0
    assert_close(out, ref, bound)
    again, _ = attend(pkv, q, cache, t, ctx, dtype, ws_byte=0x11)
    assert torch.equal(out, again)                            # whatever the workspace held


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_grow_along_the_context(pkv, dtype):
    """Every tile brings a far larger maximum, so that what was summed is rescaled each
    time; then the same keys the other way round, so that nothing after the first counts."""
    rng = np.random.default_rng(11)
    n, r, h = 700, 512, 20
    t, nb = tables_for(rng, [n, n])
    cache = latent_cache(rng, nb, r, dtype)
    rows = values(rng, (n, r + 64), dtype)
    up = np.zeros(n, np.float32)
    up[:] = np.arange(n) // 8
    if dtype == "bf16":
        rows[:, r] = (up.view(np.uint32) >> 16).astype(np.uint16)
    else:
        rows[:, r] = up
    fill(cache, t[0], rows)
    fill(cache, t[1], rows[::-1])
    q = values(rng, (2, h, r + 64), dtype, 0.1)
    q[:, :, r] = 0x4180 if dtype == "bf16" else 16.0
    start, ctx = np.arange(3), [n, n]
    ref = latent.absorbed(q, cache, t, start, ctx, 1.0, dtype)
    out, code = attend(pkv, q, cache, t, ctx, dtype, scale=1.0)
    assert code == 0
    assert_close(out, ref, absorbed_bound(q, cache, t, start, ctx, 1.0, dtype, ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_rows_come_back(pkv, dtype):
    """A weighted mean of equal rows is the row, up to the roundings of the mean itself."""
    rng = np.random.default_rng(12)
    row = values(rng, (1, 576), dtype)
    t, nb = tables_for(rng, [777])
    cache = latent_cache(rng, nb, 512, dtype)
    fill(cache, t[0], np.repeat(row, 777, 0))
    q = values(rng, (1, 9, 576), dtype)
    out, code = attend(pkv, q, cache, t, [777], dtype)
    want = widen(row, dtype)[0, :512]
    assert code == 0
    err = np.abs(out.float().cpu().numpy().astype(np.float64)[0] - want)
    assert (err <= (ROUND[dtype] + 2 * gamma(2 * 777 + 304)) * np.abs(want)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan_stay_in_their_sequence(pkv, dtype):
    """A sequence whose rows hold NaN gets NaN; its neighbours, whose tiles use the same
    buffers before and after, do not."""
    rng = np.random.default_rng(13)
    ctx = [100, 70, 100, 5]
    cache, t = batch(rng, dtype, 256, ctx)
    nan = 0x7FC0 if dtype == "bf16" else np.nan
    cache[t[1, 2], 3, :] = nan
    q = values(rng, (4, 16, 320), dtype)
    start = np.arange(5)
    good = cache.copy()
    good[t[1, 2], 3, :] = 0
    ref = latent.absorbed(q, good, t, start, ctx, SCALE, dtype)
    bound = absorbed_bound(q, good, t, start, ctx, SCALE, dtype, ref)
    ref[1] = np.nan
    out, code = attend(pkv, q, cache, t, ctx, dtype)
    assert code == 0 and torch.isnan(out[1]).all()
    assert_close(out, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fault,code", [("zero", 2), ("above", 2), ("below", 2), ("narrow", 7)])
def test_contexts_out_of_range_give_zeros(pkv, dtype, fault, code):
    rng = np.random.default_rng(14)
    ctx, new = [90, 60, 33], [2, 3, 1]
    cache, t = batch(rng, dtype, 128, ctx)
    start = np.concatenate([[0], np.cumsum(new)])
    q = values(rng, (6, 6, 192), dtype)
    ref = latent.absorbed(q, cache, t, start, ctx, SCALE, dtype)
    bound = absorbed_bound(q, cache, t, start, ctx, SCALE, dtype, ref)
    given = list(ctx)
    given[1] = {"zero": 0, "above": 91, "below": 2, "narrow": 97}[fault]
    out, got = attend(pkv, q, cache, t, given, dtype, start, most=90 if fault == "above" else 200)
    assert got == code and (out[2:5] == 0).all()
    ref[2:5] = np.nan
    assert_close(out, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("start,left", [([0, 2, 1, 3], [1]), ([1, 2, 3, 4], [0, 1]),
                                        ([0, 1, 2, 9], [2, 3]), ([0, -1, 2, 3], [0, 1])])
def test_query_layouts_that_do_not_fit(pkv, dtype, start, left):
    """Flagged; the sequences whose offsets are in order are computed, the rows of the
    others left as they were, and nothing outside touched."""
    rng = np.random.default_rng(15)
    cache, t = batch(rng, dtype, 128, [40, 50, 60])
    q = values(rng, (4, 3, 192), dtype)
    out, code = attend(pkv, q, cache, t, [40, 50, 60], dtype, start)
    assert code == 5
    if start[1] == 1 or start[0] == 1:
        for row in left:
            assert (out[row] == 7.0).all() or start[0] == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [-1, "pool"])
def test_block_ids_out_of_range_are_flagged(pkv, dtype, bad):
    rng = np.random.default_rng(16)
    ctx = [50, 90, 70]
    cache, t = batch(rng, dtype, 384, ctx)
    q = values(rng, (3, 10, 448), dtype)
    start = np.arange(4)
    ref = latent.absorbed(q, cache, t, start, ctx, SCALE, dtype)
    bound = absorbed_bound(q, cache, t, start, ctx, SCALE, dtype, ref)
    t[1, 2] = cache.shape[0] if bad == "pool" else bad
    out, code = attend(pkv, q, cache, t, ctx, dtype)
    assert code == 1
    ref[1] = np.nan
    assert_close(out, ref, bound)


def test_pool_past_32_bit_offsets(pkv):
    """Blocks at the far end of a 5 GB pool."""
    rng = np.random.default_rng(17)
    nb, r, ctx = 280000, 512, [40, 33]
    small, t = batch(rng, "bf16", r, ctx)
    q = values(rng, (2, 8, r + 64), "bf16")
    ref = latent.absorbed(q, small, t, np.arange(3), ctx, SCALE, "bf16")
    bound = absorbed_bound(q, small, t, np.arange(3), ctx, SCALE, "bf16", ref)
    pool = torch.empty((nb, 16, r + 64), dtype=torch.bfloat16, device="cuda")
    pool[nb - small.shape[0]:] = to_dev(small, "bf16")
    far = np.where(t >= 0, t + nb - small.shape[0], -1)
    desc = pkv.latent_desc(pool, r, 8)
    out = torch.empty((2, 8, r), dtype=torch.bfloat16, device="cuda")
    pkv.paged_attention_latent(out, to_dev(q, "bf16"), pool, desc, i32(far), i32(ctx), 64, SCALE)
    x = torch.empty((73, r), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((73, 64), dtype=torch.bfloat16, device="cuda")
    pkv.paged_latent_gather(x, k, pool, desc, i32(far), i32([0, 40, 73]))
    assert pkv.device_error() == 0
    assert_close(out, ref, bound)
    want = np.concatenate([latent.rows_of(small, t[s], c) for s, c in enumerate(ctx)])
    assert np.array_equal(host(x), want[:, :r]) and np.array_equal(host(k), want[:, r:])


# ------------------------------------------------------------------------------------
# streams, graphs, a run of the calls
# ------------------------------------------------------------------------------------
def test_two_calls_at_once_on_two_streams(pkv):
    """Two streams with a workspace each, over and over, give what one call gives."""
    rng = np.random.default_rng(18)
    args, want = [], []
    for ctx, h in (([3000, 900], 32), ([2500, 70, 41], 70)):
        cache, t = batch(rng, "bf16", 512, ctx)
        q = values(rng, (len(ctx), h, 576), "bf16")
        cd = to_dev(cache, "bf16")
        desc = pkv.latent_desc(cd, 512, h)
        args.append((to_dev(q, "bf16"), cd, desc, i32(t), i32(ctx), max(ctx), SCALE))
        out = torch.empty((len(ctx), h, 512), dtype=torch.bfloat16, device="cuda")
        want.append(pkv.paged_attention_latent(out, *args[-1]).clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    outs = [[torch.empty_like(w) for _ in range(10)] for w in want]
    for i in range(10):
        for a, o, s in zip(args, outs, streams):
            pkv.paged_attention_latent(o[i], *a, stream=s)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
    for o, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in o)


def test_a_step_served_from_the_device(pkv):
    """Prompts, then decode steps captured once and replayed: tables and slots from the
    requests' lengths, append with norm and rotation, absorbed attention; prompts by the
    gather, the caller's products and expanded attention.  Every step against the float64
    restatement of the whole run, over the rows as the cache holds them."""
    rng = np.random.default_rng(19)
    dtype, r, h, d, nb = "bf16", 256, 12, 128, 60
    lens, steps = [70, 5, 33], 4
    tab, w = rope.rope_table(512, 64), values(rng, (r,), dtype)
    wk, wv = (to_dev(values(rng, (h, d, r), dtype, r ** -0.5), dtype) for _ in range(2))
    n, total = len(lens), sum(lens)
    tables = pkv.DeviceTables.create(nb, 16, n, 16, rng.permutation(nb))
    cache = to_dev(latent_cache(rng, nb, r, dtype), dtype)
    desc = pkv.latent_desc(cache, r, h)
    tabd, wd = to_dev(tab), to_dev(w, dtype)
    scale = (d + 64) ** -0.5

    def step_buffers(tokens):
        def new(*s, dt=torch.int32):
            return torch.empty(s, dtype=dt, device="cuda")
        return dict(t=new(n, 16), start=new(n + 1), slots=new(tokens, dt=torch.int64),
                    pos=new(tokens))

    def run(b, ctx, new_lens, down, q):
        """Append a step's tokens; returns the rotated queries [T, H, d + 64]."""
        pkv.pkv_tables_step(tables, None, ctx, new_lens, b["t"], ctx, b["start"], b["slots"],
                            b["pos"])
        rot = torch.cat([q[..., :d], torch.empty_like(q[..., d:])], -1)
        pkv.paged_latent_append(down[:, :r], down[:, r:], b["slots"], b["pos"], tabd, cache, desc,
                                wd, 1e-6, q[..., d:], rot[..., d:], True)
        return rot

    # prompts, expanded
    ctx, b = i32([0] * n), step_buffers(total)
    down = to_dev(values(rng, (total, r + 64), dtype), dtype)
    q = to_dev(values(rng, (total, h, d + 64), dtype), dtype)
    rot = run(b, ctx, i32(lens), down, q)
    rows, keys = (torch.empty((total, x), dtype=cache.dtype, device="cuda") for x in (r, 64))
    pkv.paged_latent_gather(rows, keys, cache, desc, b["t"], b["start"])
    k, v = (torch.einsum("tr,hdr->thd", rows, m).contiguous() for m in (wk, wv))
    out = torch.empty((total, h, d), dtype=cache.dtype, device="cuda")
    pkv.pkv_attention_expanded(out, rot, k, v, keys, b["start"], b["start"], max(lens))
    assert pkv.device_error() == 0
    from tests.latent_checks import expanded_bound
    starts = np.concatenate([[0], np.cumsum(lens)])
    args = (host(rot), host(k), host(v), host(keys), starts, starts, scale, dtype)
    ref = latent.expanded(*args)
    assert_close(out, ref, expanded_bound(*args, ref))
    # the cache holds what the oracle's append gives, up to the norm's rounding
    a, kk, done = latent.append(host(down)[:, :r], np.ascontiguousarray(host(down)[:, r:]),
                                host(b["slots"]), host(b["pos"]), tab, 16, nb, dtype, w, 1e-6, True)
    got = host(cache)
    assert np.array_equal(got[..., r:][done], kk[done])
    assert (np.abs(widen(got[..., :r], dtype) - a)[done]
            <= ((gamma(r + 8) + ROUND[dtype]) * np.abs(a))[done] + 1e-30).all()

    # decode, absorbed: one captured step, replayed
    b = step_buffers(n)
    down_in = torch.empty((n, r + 64), dtype=cache.dtype, device="cuda")
    q_in = torch.empty((n, h, d + 64), dtype=cache.dtype, device="cuda")
    absorbed = torch.empty((n, h, r + 64), dtype=cache.dtype, device="cuda")
    lat = torch.empty((n, h, r), dtype=cache.dtype, device="cuda")
    ws = pkv.workspace(pkv.latent_workspace_bytes(desc, n, n, 256))
    pkv.paged_attention_latent(lat, absorbed.zero_(), cache, desc, b["t"].zero_(), i32([1] * n), 256,
                               scale, ws=ws)              # first call outside the capture
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.pkv_tables_step(tables, None, ctx, None, b["t"], ctx, b["start"], b["slots"], b["pos"])
        absorbed[..., :r] = torch.einsum("thd,hdr->thr", q_in[..., :d], wk)
        pkv.paged_latent_append(down_in[:, :r], down_in[:, r:], b["slots"], b["pos"], tabd, cache,
                                desc, wd, 1e-6, q_in[..., d:], absorbed[..., r:], True)
        pkv.paged_attention_latent(lat, absorbed, cache, desc, b["t"], ctx, 256, scale, ws=ws)
    for i in range(steps):
        down_in.copy_(to_dev(values(rng, (n, r + 64), dtype), dtype))
        q_in.copy_(to_dev(values(rng, (n, h, d + 64), dtype), dtype))
        graph.replay()
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        c = [x + i + 1 for x in lens]
        assert ctx.tolist() == c
        args = (host(absorbed), host(cache), host(b["t"]), np.arange(n + 1), c, scale, dtype)
        ref = latent.absorbed(*args)
        assert_close(lat, ref, absorbed_bound(*args, ref))


def test_graphs_with_a_workspace_each(pkv):
    """Two captured calls whose lengths change between replays."""
    rng = np.random.default_rng(20)
    cache, t = batch(rng, "bf16", 128, [600, 600])
    cd, td = to_dev(cache, "bf16"), i32(t)
    graphs = []
    for h in (8, 40):
        q = values(rng, (2, h, 192), "bf16")
        desc = pkv.latent_desc(cd, 128, h)
        ctx, out = i32([1, 1]), torch.empty((2, h, 128), dtype=torch.bfloat16, device="cuda")
        ws = pkv.workspace(pkv.latent_workspace_bytes(desc, 2, 2, 600))
        call = (out, to_dev(q, "bf16"), cd, desc, td, ctx, 600, SCALE, None, ws)
        pkv.paged_attention_latent(*call)
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            pkv.paged_attention_latent(*call)
        graphs.append((g, s, q, ctx, out, call))             # what was captured stays alive
    for lens in ([600, 3], [17, 599], [0, 128]):
        for g, s, q, ctx, out, _ in graphs:
            ctx.copy_(i32(lens))
        torch.cuda.synchronize()
        for g, s, q, ctx, out, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert pkv.device_error() == (2 if 0 in lens else 0)
        for g, s, q, ctx, out, _ in graphs:
            for i, c in enumerate(lens):
                if c == 0:
                    assert (out[i] == 0).all()
                    continue
                args = (q[i:i + 1], cache, t[i:i + 1], [0, 1], [c], SCALE, "bf16")
                ref = latent.absorbed(*args)
                assert_close(out[i:i + 1], ref, absorbed_bound(*args, ref))


def test_binding_refuses_on_the_gpu(pkv):
    c = torch.zeros((4, 16, 192), device="cuda")
    desc = pkv.latent_desc(c, 128, 2)
    q, out = torch.zeros((1, 2, 192), device="cuda"), torch.zeros((1, 2, 128), device="cuda")
    t, ctx = i32([[0]]), i32([5])
    ok = (out, q, c, desc, t, ctx, 16, SCALE)
    pkv.paged_attention_latent(*ok)
    for at, wrong in ((0, out[..., :64]), (1, q[:, :1]), (1, q.double()), (2, c[:2]),
                      (1, q.transpose(0, 1)), (4, t.long()), (5, ctx.cpu())):
        args = list(ok)
        args[at] = wrong
        with pytest.raises((TypeError, ValueError)):
            pkv.paged_attention_latent(*args)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_attention_latent(*ok, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    x, k = torch.zeros((1, 128), device="cuda"), torch.zeros((1, 64), device="cuda")
    slots, pos, tab = torch.zeros(1, dtype=torch.int64).cuda(), i32([0]), torch.zeros((4, 64)).cuda()
    with pytest.raises(ValueError, match="contiguous"):
        pkv.paged_latent_append(torch.zeros((128, 1), device="cuda").t().expand(1, 128)[:, ::1]
                                .as_strided((1, 128), (128, 0)), k, slots, pos, tab, c, desc)
    with pytest.raises(ValueError, match="together"):
        pkv._native().latent_append(x, k, slots, pos, tab, c, desc, None, 0.0, None, q[..., :64],
                                    False, None)
    with pytest.raises(pkv.PagedKVError):                     # rows that do not start on 16 bytes
        pkv.paged_latent_append(torch.zeros((2, 130), device="cuda")[:, 1:129],
                                torch.zeros((2, 64), device="cuda"), slots.expand(2).contiguous(),
                                pos.expand(2).contiguous(), tab, c, desc)
    torch.cuda.synchronize()
    assert pkv.device_error() == 0


def test_single_precision_units_of_32_rows_cut_over_ctas(pkv):
    """72 rows a sequence of the longest vectors, a context that many CTAs share."""
    rng = np.random.default_rng(23)
    ctx, start = [2500, 19, 3], [0, 2, 3, 4]
    cache, t = batch(rng, "f32", 512, ctx)
    q = values(rng, (4, 36, 576), "f32")
    args = (q, cache, t, start, ctx, SCALE, "f32")
    ref = latent.absorbed(*args)
    out, code = attend(pkv, q, cache, t, ctx, "f32", start)
    assert code == 0
    assert_close(out, ref, absorbed_bound(*args, ref))
