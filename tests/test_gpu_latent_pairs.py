"""GPU: latent attention of sequences with more than 64 (token, head) rows, which pairs of
CTAs take 128 rows and 128 keys at a time, against the float64 restatement."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import latent  # noqa: E402
from oracle.numerics import widen  # noqa: E402
from tests.gpu_parity import gamma  # noqa: E402
from tests.latent_checks import absorbed_bound, assert_close, fill, latent_cache  # noqa: E402
from tests.sparse_checks import ROUND, i32, tables_for, to_dev, values  # noqa: E402
from tests.test_gpu_latent import SCALE, attend, batch, pkv  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def check(pkv, q, cache, t, ctx, start=None, scale=SCALE):  # noqa: F811
    rows = np.arange(len(ctx) + 1) if start is None else start
    ref = latent.absorbed(q, cache, t, rows, ctx, scale, "bf16")
    out, code = attend(pkv, q, cache, t, ctx, "bf16", start, scale=scale)
    assert code == 0
    assert_close(out, ref, absorbed_bound(q, cache, t, rows, ctx, scale, "bf16", ref))
    return out


@pytest.mark.parametrize("r", [128, 256, 384, 512])
@pytest.mark.parametrize("h", [65, 96, 97, 128])
def test_one_token_a_sequence(pkv, r, h):  # noqa: F811
    """Contexts around the edges of blocks, of 32 values' keys, of a CTA's 64 keys and of
    tiles; rows of the pool that no token was written to hold NaN."""
    ctx = [1, 128, 15, 129, 16, 17, 127, 31, 32, 33, 49, 63, 64, 65, 112, 256, 300]
    rng = np.random.default_rng(r + h)
    cache, t = batch(rng, "bf16", r, ctx)
    check(pkv, values(rng, (len(ctx), h, r + 64), "bf16"), cache, t, ctx)


@pytest.mark.parametrize("r,h,new,ctx", [
    (512, 24, [3, 4, 0, 6], [130, 129, 9, 6]),
    (128, 100, [2, 1, 3], [257, 33, 3]),
    (256, 129, [1, 1], [140, 5]),
    (384, 9, [40, 1], [400, 128]),                            # 360 rows and 9
    (512, 300, [2], [131]),
])
def test_several_tokens_a_sequence(pkv, r, h, new, ctx):  # noqa: F811
    """Causal limits inside a tile and in front of it, rows that end in the first CTA's half,
    padding rows behind the last sequence."""
    rng = np.random.default_rng(h)
    cache, t = batch(rng, "bf16", r, ctx)
    start = np.concatenate([[0], np.cumsum(new)])
    out = check(pkv, np.concatenate([values(rng, (start[-1], h, r + 64), "bf16"),
                                     np.full((2, h, r + 64), 0x7FC0, np.uint16)]),
                cache, t, ctx, start)
    assert (out[start[-1]:] == 7.0).all()


@pytest.mark.parametrize("r,h,ctx", [(512, 128, [7000, 3, 700]), (128, 80, [20] * 300)])
def test_long_contexts_and_many_sequences(pkv, r, h, ctx):  # noqa: F811
    """Units cut over many pairs and joined; several units a pair; twice the same."""
    rng = np.random.default_rng(len(ctx))
    cache, t = batch(rng, "bf16", r, ctx)
    q = values(rng, (len(ctx), h, r + 64), "bf16")
    out = check(pkv, q, cache, t, ctx)
    again, _ = attend(pkv, q, cache, t, ctx, "bf16", ws_byte=0x11)
    assert torch.equal(out, again)


def test_scores_that_grow_along_the_context(pkv):  # noqa: F811
    rng = np.random.default_rng(11)
    n, r, h = 900, 512, 70
    t, nb = tables_for(rng, [n, n])
    cache = latent_cache(rng, nb, r, "bf16")
    rows = values(rng, (n, r + 64), "bf16")
    up = (np.arange(n) // 8).astype(np.float32)
    rows[:, r] = (up.view(np.uint32) >> 16).astype(np.uint16)
    fill(cache, t[0], rows)
    fill(cache, t[1], rows[::-1])
    q = values(rng, (2, h, r + 64), "bf16", 0.1)
    q[:, :, r] = 0x4180
    check(pkv, q, cache, t, [n, n], scale=1.0)


def test_equal_rows_come_back(pkv):  # noqa: F811
    rng = np.random.default_rng(12)
    row = values(rng, (1, 448), "bf16")
    t, nb = tables_for(rng, [777])
    cache = latent_cache(rng, nb, 384, "bf16")
    fill(cache, t[0], np.repeat(row, 777, 0))
    out, code = attend(pkv, values(rng, (1, 99, 448), "bf16"), cache, t, [777], "bf16")
    want = widen(row, "bf16")[0, :384]
    assert code == 0
    err = np.abs(out.float().cpu().numpy().astype(np.float64)[0] - want)
    assert (err <= (ROUND["bf16"] + 2 * gamma(2 * 777 + 304)) * np.abs(want)).all()


@pytest.mark.parametrize("fault,code", [("nan", 0), ("id", 1), ("zero", 2), ("above", 2), ("narrow", 7)])
def test_what_is_wrong_stays_in_its_sequence(pkv, fault, code):  # noqa: F811
    rng = np.random.default_rng(13)
    ctx, h, r = [100, 170, 300, 5], 90, 256
    cache, t = batch(rng, "bf16", r, ctx)
    q = values(rng, (4, h, r + 64), "bf16")
    start = np.arange(5)
    ref = latent.absorbed(q, cache, t, start, ctx, SCALE, "bf16")
    bound = absorbed_bound(q, cache, t, start, ctx, SCALE, "bf16", ref)
    bad = 1
    if fault == "nan":
        cache[t[1, 2], 3, :] = 0x7FC0
    elif fault == "id":
        t[1, 9] = cache.shape[0]
    elif fault == "narrow":
        bad, t = 2, t[:, :12]
        # (the other sequences fit into 12 blocks)
    else:
        ctx[1] = 0 if fault == "zero" else 301
    ref[bad] = np.nan
    out, got = attend(pkv, q, cache, t, ctx, "bf16", most=300)
    assert got == code
    assert_close(out, ref, bound)
    if fault == "nan":
        assert torch.isnan(out[bad]).all()
    elif fault != "id":
        assert (out[bad] == 0).all()


def test_a_captured_call_replayed_with_other_lengths(pkv):  # noqa: F811
    """Two graphs on two streams, each with its own workspace."""
    rng = np.random.default_rng(20)
    cache, t = batch(rng, "bf16", 512, [600, 600])
    cd, td = to_dev(cache, "bf16"), i32(t)
    graphs = []
    for h in (72, 128):
        q = values(rng, (2, h, 576), "bf16")
        desc = pkv.latent_desc(cd, 512, h)
        ctx, out = i32([1, 1]), torch.empty((2, h, 512), dtype=torch.bfloat16, device="cuda")
        ws = pkv.workspace(pkv.latent_workspace_bytes(desc, 2, 2, 600))
        call = (out, to_dev(q, "bf16"), cd, desc, td, ctx, 600, SCALE, None, ws)
        pkv.paged_attention_latent(*call)
        torch.cuda.synchronize()
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=s):
            pkv.paged_attention_latent(*call)
        graphs.append((g, s, q, ctx, out, call))             # what was captured stays alive
    for lens in ([600, 3], [17, 599], [128, 256]):
        for g, s, q, ctx, out, _ in graphs:
            ctx.copy_(i32(lens))
        torch.cuda.synchronize()
        for g, s, q, ctx, out, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        for g, s, q, ctx, out, _ in graphs:
            args = (q, cache, t, [0, 1, 2], lens, SCALE, "bf16")
            ref = latent.absorbed(*args)
            assert_close(out, ref, absorbed_bound(*args, ref))
