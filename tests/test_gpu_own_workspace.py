"""GPU: calls that take their own workspace, on a stream beside a busy current one."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sparse  # noqa: E402
from tests.sparse_checks import i32, tables_for, to_dev, values  # noqa: E402

pytestmark = pytest.mark.gpu

CALLS = 6


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


def _beside_a_busy_stream(nbytes, call):
    """call(i, stream) CALLS times on a side stream.  Before each, the current stream
    gets a few milliseconds of work on memory of a workspace's size, which the
    program has given back by the time of the call: it is filled, read at the end of
    that work (what was filled has to be there still), and written again."""
    a = torch.randn((8192, 8192), dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(CALLS):
        temporary = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")
        kept = torch.empty_like(temporary)
        torch.cuda.synchronize()
        temporary.fill_(0xA5)
        for _ in range(5):
            torch.mm(a, a, out=b)
        kept.copy_(temporary)
        temporary.fill_(0xFF)
        del temporary
        call(i, side)
        torch.cuda.synchronize()
        assert (kept == 0xA5).all()


def test_selection_beside_a_busy_stream(pkv):
    rng = np.random.default_rng(30)
    ctx = [9000, 7000]
    t, nb = tables_for(rng, ctx)
    mid, half = rng.normal(0, 25, (nb, 2, 128)), np.abs(rng.normal(30, 8, (nb, 2, 128)))
    bounds = np.clip(np.rint(np.stack([mid + half, mid - half], 2)), -127, 127).astype(np.int8)
    exps = rng.integers(-7, -4, (nb, 2)).astype(np.int8)
    q = values(rng, (2, 4, 128), "bf16")
    desc = pkv.CacheDesc(pkv.PKV_BF16, nb, 16, 2, 4, 128)
    args = [to_dev(q, "bf16"), to_dev(bounds), to_dev(exps), desc, i32(t), i32(ctx), max(ctx), 1, 1]
    sel = [torch.full((2, 2, 20), -9, dtype=torch.int32, device="cuda") for _ in range(CALLS)]
    _beside_a_busy_stream(pkv.select_workspace_bytes(desc, 2, max(ctx)),
                          lambda i, side: pkv.pkv_select_blocks(sel[i], *args, stream=side))
    assert pkv.device_error() == 0
    ref = sparse.select(q, bounds, exps, t, [0, 1, 2], ctx, 16, 20, 1, 1, "bf16")
    for s in sel:
        assert np.array_equal(s.cpu().numpy(), ref)


@pytest.mark.parametrize("kind", ["decode", "varlen", "int8"])
def test_dense_attention_beside_a_busy_stream(pkv, kind):
    """The same lists of splits and partial results as with a workspace of the
    caller's, bit for bit."""
    rng = np.random.default_rng(31)
    ctx = [9000, 7000, 600]
    t, nb = tables_for(rng, ctx)
    td, cd, start = i32(t), i32(ctx), i32([0, 1, 2, 3])
    q = to_dev(values(rng, (3, 8, 128), "bf16"), "bf16")
    k, v = (to_dev(values(rng, (sum(ctx), 2, 128), "bf16"), "bf16") for _ in range(2))
    slots = torch.cat([td[s, torch.arange(n, device="cuda") // 16].long() * 16 +
                       torch.arange(n, device="cuda") % 16 for s, n in enumerate(ctx)])
    if kind == "int8":
        cache = pkv.Int8Cache(nb, 2, 16, 128, 8)
        pkv.paged_kv_append_int8(k, v, slots, cache)
        need = pkv.decode_workspace_bytes(cache.desc, 3, max(ctx))
    else:
        kc, vc = (torch.zeros((nb, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
        desc = pkv.cache_desc(kc, 8)
        pkv.paged_kv_append(k, v, slots, kc, vc, desc)
        need = (pkv.decode_workspace_bytes(desc, 3, max(ctx)) if kind == "decode" else
                pkv.varlen_workspace_bytes(desc, 3, 3, 1, max(ctx)))

    def call(out, **kw):
        if kind == "int8":
            pkv.paged_attention_decode_int8(out, q, cache, td, cd, max(ctx), **kw)
        elif kind == "decode":
            pkv.paged_attention_decode(out, q, kc, vc, desc, td, cd, max(ctx), **kw)
        else:
            pkv.paged_attention_varlen(out, q, kc, vc, desc, td, start, cd, 1, max(ctx), **kw)

    ref, outs = torch.empty_like(q), [torch.empty_like(q) for _ in range(CALLS)]
    call(ref, ws=pkv.workspace(need))
    _beside_a_busy_stream(need, lambda i, side: call(outs[i], stream=side))
    assert pkv.device_error() == 0
    for out in outs:
        assert torch.equal(out, ref)
