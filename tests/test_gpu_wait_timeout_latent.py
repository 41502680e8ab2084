"""GPU: waits of the latent and the expanded attention's pipelines that run out.

As for the decode kernel, a copy of the library with a 1 ms limit whose loaders leave out a
CTA's fourth tile (nothing is copied or expected for it): the products' issuer runs out of
time, and with it every role that waits for it, each within its own limit.  The kernel ends,
the error word says why, nothing outside the output and the workspace is written, and the
product library's next call on the same context gives the bits that it gave before."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.sparse_checks import i32, to_dev, values  # noqa: E402
from tests.test_gpu_expanded import Case  # noqa: E402
from tests.test_gpu_latent import SCALE, batch, pkv  # noqa: E402, F401
from tests.test_gpu_sparse_layouts import fenced  # noqa: E402
from tests.test_gpu_wait_timeout import WAIT_TEST_DEFINES  # noqa: E402

pytestmark = pytest.mark.gpu

WAIT_TIMEOUT = 6


@pytest.fixture(scope="module")
def slow(pkv):  # noqa: F811
    """The copy of the library, with the product's prototypes."""
    from paged_kv_cache_51_gb300 import _build

    T = ctypes.CDLL(_build.build_variant("waittest", WAIT_TEST_DEFINES))
    for name in ("paged_attention_latent", "pkv_attention_expanded", "pkv_device_error"):
        f, g = getattr(T, name), getattr(pkv.lib(), name)
        f.restype, f.argtypes = g.restype, g.argtypes
    code = ctypes.c_int32()
    assert T.pkv_device_error(ctypes.byref(code), 1) == 0
    return T


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def check(pkv, slow, good, out, ws, call):  # noqa: F811
    """good(): the product's call; call(out, ws): the copy's."""
    want = good()
    assert pkv.device_error() == 0
    out, out_whole = fenced(out)
    ws, ws_whole = fenced(ws)
    assert call(out, ws) == 0
    code = ctypes.c_int32()
    assert slow.pkv_device_error(ctypes.byref(code), 1) == 0      # synchronizes the device
    assert code.value == WAIT_TIMEOUT
    assert out_whole() and ws_whole()
    again = good()
    assert pkv.device_error() == 0
    assert torch.equal(again, want)


@pytest.mark.parametrize("r,h", [(512, 40), (128, 16), (512, 128), (128, 80)])
def test_latent(pkv, slow, r, h):  # noqa: F811
    """Single CTAs and pairs, rings of the longest and the shortest vectors; every CTA has
    more than four tiles."""
    rng = np.random.default_rng(h)
    ctx = [8000, 7990, 8100, 8003, 7777, 8000, 8001, 8192]
    cache, t = batch(rng, "bf16", r, ctx)
    q, c = to_dev(values(rng, (8, h, r + 64), "bf16"), "bf16"), to_dev(cache, "bf16")
    desc, td, cd = pkv.latent_desc(c, r, h), i32(t), i32(ctx)
    need = pkv.latent_workspace_bytes(desc, 8, 8, 8192)

    def good():
        out = torch.empty((8, h, r), dtype=q.dtype, device="cuda")
        return pkv.paged_attention_latent(out, q, c, desc, td, cd, 8192, SCALE)

    def call(out, ws):
        return slow.paged_attention_latent(
            ptr(out), ptr(q), ptr(c), ctypes.byref(desc), ptr(td), td.shape[1], None, ptr(cd), 8, 8,
            8192, SCALE, ptr(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))

    check(pkv, slow, good, torch.zeros((8, h, r), dtype=q.dtype, device="cuda"),
          torch.zeros(need, dtype=torch.uint8, device="cuda"), call)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,new,keys", [(8, [300, 500], [900, 1000]), (50, [20], [2000]), (1, [16], [4000])])
def test_expanded(pkv, slow, d, h, new, keys):  # noqa: F811
    """One CTA a unit, clusters of two and of four; every CTA has more than four tiles."""
    c = Case(np.random.default_rng(h), "bf16", h, d, new, keys, pad=0)
    q, kv, r = (to_dev(x, "bf16") for x in (c.q, c.kv, c.r))
    k, v, qs, ks = kv[..., :d], kv[..., d:], i32(c.qs), i32(c.ks)
    desc = pkv.ExpandedDesc(pkv.PKV_BF16, h, d, 64, h * 2 * d, 2 * d, h * 2 * d, 2 * d)
    need = pkv.lib().pkv_expanded_workspace_bytes(ctypes.byref(desc), len(new), q.shape[0])
    shape = (q.shape[0], h, d)

    def good():
        out = torch.empty(shape, dtype=q.dtype, device="cuda")
        return pkv.pkv_attention_expanded(out, q, k, v, r, qs, ks, c.most)

    def call(out, ws):
        return slow.pkv_attention_expanded(
            ptr(out), ptr(q), ptr(k), ptr(v), ptr(r), ctypes.byref(desc), ptr(qs), ptr(ks), len(new),
            q.shape[0], k.shape[0], c.most, c.scale, ptr(ws), ws.numel(),
            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))

    check(pkv, slow, good, torch.zeros(shape, dtype=q.dtype, device="cuda"),
          torch.zeros(need, dtype=torch.uint8, device="cuda"), call)
