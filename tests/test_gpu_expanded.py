"""GPU: attention over expanded keys against the float64 restatement."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import latent  # noqa: E402
from tests.latent_checks import assert_close, expanded_bound  # noqa: E402
from tests.sparse_checks import i32, to_dev, values  # noqa: E402
from tests.test_gpu_sparse_layouts import fenced  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


class Case:
    """Queries, keys and values of a few sequences; keys and values side by side, as the
    expansion leaves them, with NaN in `pad` rows behind the last sequence's."""

    def __init__(self, rng, dtype, h, d, new, keys, pad=2, scale=None, k_scale=1.0):
        self.dtype, self.h, self.d = dtype, h, d
        self.qs, self.ks = (np.concatenate([[0], np.cumsum(x)]) for x in (new, keys))
        nan = 0x7FC0 if dtype == "bf16" else np.nan
        self.q = values(rng, (self.qs[-1] + pad, h, d + 64), dtype)
        self.kv = values(rng, (self.ks[-1] + pad, h, 2 * d), dtype, k_scale)
        self.r = values(rng, (self.ks[-1] + pad, 64), dtype)
        self.kv[self.ks[-1]:], self.r[self.ks[-1]:] = nan, nan
        self.most = max(new)
        self.scale = scale or (d + 64) ** -0.5

    def oracle(self):
        a = (self.q, np.ascontiguousarray(self.kv[..., :self.d]),
             np.ascontiguousarray(self.kv[..., self.d:]), self.r, self.qs, self.ks, self.scale,
             self.dtype)
        ref = latent.expanded(*a)
        return ref, expanded_bound(*a, ref)

    def run(self, pkv, ws_byte=0xFF, q_start=None, k_start=None, most=None, offset=0, **kw):
        kv, qd = to_dev(self.kv, self.dtype), to_dev(self.q, self.dtype)
        rd = to_dev(self.r, self.dtype)
        shape = (self.q.shape[0], self.h, self.d)
        out, whole = fenced(torch.full(shape, 7.0, dtype=kv.dtype, device="cuda"),
                            before=4096 + offset)
        args = (out, qd, kv[..., :self.d], kv[..., self.d:], rd,
                i32(self.qs if q_start is None else q_start),
                i32(self.ks if k_start is None else k_start), most or self.most, self.scale)
        need = pkv._native().attention_expanded(*args, None, None)
        ws, ws_whole = fenced(torch.full((need,), ws_byte, dtype=torch.uint8, device="cuda"))
        pkv.pkv_attention_expanded(*args, ws=ws, **kw)
        code = pkv.device_error()
        assert whole() and ws_whole()
        return out, code

    def check(self, pkv):
        ref, bound = self.oracle()
        out, code = self.run(pkv)
        assert code == 0
        assert_close(out, ref, bound)
        assert (out[self.qs[-1]:] == 7.0).all()
        return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,new,keys", [
    (1, [1], [1]),
    (3, [1, 1, 1], [1, 130, 17]),
    (2, [5, 0, 127, 3], [5, 9, 127, 200]),
    (1, [128, 129], [128, 129]),
    (2, [300], [301]),
    (5, [40, 1, 64], [300, 64, 64]),
])
def test_ragged_batches(pkv, dtype, d, h, new, keys):
    Case(np.random.default_rng(h + d), dtype, h, d, new, keys).check(pkv)


@pytest.mark.parametrize("dtype,d,h,new,keys", [
    ("bf16", 128, 2, [700, 257, 255], [900, 257, 511]),
    ("bf16", 64, 3, [513, 40], [513, 1300]),
    ("f32", 128, 2, [400], [650]),
    ("f32", 64, 4, [65, 200], [65, 333]),
    ("bf16", 128, 160, [30, 200], [30, 333]),     # more units than SMs, of both streams and one
])
def test_longer_prompts_and_chunks(pkv, dtype, d, h, new, keys):
    """Several units a sequence; twice, whatever the workspace held."""
    c = Case(np.random.default_rng(h), dtype, h, d, new, keys)
    out = c.check(pkv)
    again, _ = c.run(pkv, ws_byte=0x11)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,new,keys", [
    (1, [1], [1100]),
    (3, [16], [2000]),                            # a CTA of each cluster without tiles of its own
    (2, [300, 5, 0, 129], [2500, 613, 600, 640]),
    (1, [1300], [1200]),                          # queries that see no key
    (9, [1, 1, 1, 40], [4100, 1, 2, 41]),         # units without keys for every CTA
    (25, [300], [1030]),                          # by two CTAs
    (1, [1025], [1025]),
])
def test_few_units_share_a_cluster(pkv, d, h, new, keys):
    """So few units that four CTAs take the keys of each, twice the same."""
    c = Case(np.random.default_rng(h + d), "bf16", h, d, new, keys)
    out = c.check(pkv)
    again, _ = c.run(pkv, ws_byte=0x11)
    assert torch.equal(out, again)


@pytest.mark.parametrize("d", [64, 128])
def test_single_precision_with_units_for_every_sm(pkv, d):
    """So many rows that a CTA takes 64 of them alone (fewer are shared by a cluster)."""
    Case(np.random.default_rng(d), "f32", 110, d, [180, 1], [200, 90]).check(pkv)


@pytest.mark.parametrize("d", [64, 128])
def test_single_precision_long_prompts(pkv, d):
    """Prompts of 512 tokens and more on average, a unit that ends inside its rows."""
    Case(np.random.default_rng(d), "f32", 20, d, [530, 500], [560, 500]).check(pkv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,keys", [([10], [4]), ([300, 7], [20, 0]), ([3, 260, 2], [0, 131, 2]),
                                      ([5], [0])])
def test_queries_that_see_no_key_are_zero(pkv, dtype, d, new, keys):
    c = Case(np.random.default_rng(d), dtype, 2, d, new, keys, pad=0 if sum(keys) == 0 else 2)
    out = c.check(pkv)
    at = 0
    for m, n in zip(new, keys):
        if m > n:
            assert (out[at:at + m - n] == 0).all()
        at += m


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_keys_at_all(pkv, dtype):
    c = Case(np.random.default_rng(1), dtype, 2, 128, [5, 3], [0, 0], pad=0)
    out, code = c.run(pkv)
    assert code == 0 and (out == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_neighbours_nan_does_not_reach_a_sequence(pkv, dtype, d):
    """The rows of the next sequence lie in a tile's tail; a NaN there is its own."""
    c = Case(np.random.default_rng(2), dtype, 2, d, [40, 30, 50], [40, 90, 50])
    ref, bound = c.oracle()
    nan = 0x7FC0 if dtype == "bf16" else np.nan
    c.kv[41:60], c.r[41:60], c.q[45] = nan, nan, nan
    out, code = c.run(pkv)
    assert code == 0 and torch.isnan(out[60:70]).all()
    ref[40:70] = np.nan
    assert_close(out, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_grow_along_the_keys(pkv, dtype, d):
    """Each tile's maximum lies far above the last one's: the output so far is rescaled."""
    rng = np.random.default_rng(3)
    c = Case(rng, dtype, 2, d, [200], [800], scale=1.0, k_scale=0.1)
    up = (np.arange(c.r.shape[0]) // 16).astype(np.float32)
    c.r[:, 0] = (up.view(np.uint32) >> 16).astype(np.uint16) if dtype == "bf16" else up
    c.q[:, :, d] = 0x4180 if dtype == "bf16" else 16.0
    c.kv[c.ks[-1]:] = 0x7FC0 if dtype == "bf16" else np.nan
    c.check(pkv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts_of_keys_and_values(pkv, dtype):
    """Tensors of their own, heads before tokens, one head alone, an output that begins on
    16 bytes only."""
    rng = np.random.default_rng(4)
    c = Case(rng, dtype, 3, 128, [50, 140], [60, 140], pad=0)
    ref, bound = c.oracle()
    kv, q, r = (to_dev(x, dtype) for x in (c.kv, c.q, c.r))
    k, v = kv[..., :128], kv[..., 128:]
    for kk, vv in ((k.contiguous(), v.contiguous()),
                   (k.permute(1, 0, 2).contiguous().permute(1, 0, 2),
                    v.permute(1, 0, 2).contiguous().permute(1, 0, 2))):
        out = torch.empty_like(q[..., :128])
        out = pkv.pkv_attention_expanded(torch.empty(out.shape, dtype=q.dtype, device="cuda"), q, kk,
                                         vv, r, i32(c.qs), i32(c.ks), c.most)
        assert pkv.device_error() == 0
        assert_close(out, ref, bound)
    one = pkv.pkv_attention_expanded(
        torch.empty((c.q.shape[0], 1, 128), dtype=q.dtype, device="cuda"), q[:, 1:2].contiguous(),
        k[:, 1:2], v[:, 1:2], r, i32(c.qs), i32(c.ks), c.most)
    assert_close(one, ref[:, 1:2], bound[:, 1:2])
    out, code = c.run(pkv, offset=16)
    assert code == 0
    assert_close(out, ref, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_start,k_start,most,left", [
    ([0, 20, 10, 60], None, None, None),
    ([0, 20, 40, 200], None, None, range(40, 60)),
    (None, [0, 30, 20, 90], None, range(20, 40)),
    (None, [0, 30, 60, 500], None, range(40, 60)),
    (None, None, 19, range(60)),
    ([1, 20, 40, 60], None, None, range(20)),
    ([0, 20, 40, 60], [-1, 30, 60, 90], None, range(20)),
])
def test_layouts_that_do_not_fit(pkv, dtype, q_start, k_start, most, left):
    """Flagged; those sequences' rows are left as they were and nothing outside touched."""
    c = Case(np.random.default_rng(5), dtype, 2, 128, [20, 20, 20], [30, 30, 30], pad=0)
    out, code = c.run(pkv, q_start=q_start, k_start=k_start, most=most)
    assert code == 5
    if left is not None:
        assert (out[list(left)] == 7.0).all()


def test_streams_and_replays(pkv):
    """Captured once, replayed with other offsets, beside an eager call on another stream."""
    rng = np.random.default_rng(6)
    c = Case(rng, "bf16", 4, 128, [100, 60, 140], [180, 60, 200], pad=0)
    kv, q, r = (to_dev(x, "bf16") for x in (c.kv, c.q, c.r))
    qs, ks = i32(c.qs), i32(c.ks)
    out = torch.empty((300, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = pkv.workspace(1 << 16)
    call = (q, kv[..., :128], kv[..., 128:], r)
    pkv.pkv_attention_expanded(out, *call, qs, ks, 300, ws=ws)
    torch.cuda.synchronize()
    g, s, side = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        pkv.pkv_attention_expanded(out, *call, qs, ks, 300, ws=ws)
    for new, keys in (([100, 60, 140], [180, 60, 200]), ([0, 300, 0], [0, 440, 0]),
                      ([1, 1, 298], [100, 1, 339])):
        c.qs, c.ks = (np.concatenate([[0], np.cumsum(x)]) for x in (new, keys))
        qs.copy_(i32(c.qs))
        ks.copy_(i32(c.ks))
        torch.cuda.synchronize()
        eager = [torch.empty_like(out) for _ in range(4)]
        with torch.cuda.stream(s):
            g.replay()
        for e in eager:
            pkv.pkv_attention_expanded(e, *call, qs, ks, 300, stream=side)
        torch.cuda.synchronize()
        assert pkv.device_error() == 0
        ref, bound = c.oracle()
        assert_close(out, ref, bound)
        assert all(torch.equal(e, out) for e in eager)


def test_binding_refuses_on_the_gpu(pkv):
    q = torch.zeros((4, 2, 128), device="cuda")
    k, r, s = torch.zeros((4, 2, 64), device="cuda"), torch.zeros((4, 64), device="cuda"), i32([0, 4])
    out = torch.zeros((4, 2, 64), device="cuda")
    ok = (out, q, k, k, r, s, s, 4)
    pkv.pkv_attention_expanded(*ok)
    for at, wrong in ((0, out[:3]), (1, q[..., :64]), (2, k[:3]), (2, k.bfloat16()), (3, k[..., :32]),
                      (4, r[:3]), (5, s.long()), (6, i32([0, 2, 4])), (2, k.transpose(1, 2))):
        args = list(ok)
        args[at] = wrong
        with pytest.raises((TypeError, ValueError, pkv.PagedKVError)):
            pkv.pkv_attention_expanded(*args)
    with pytest.raises(pkv.PagedKVError):                     # heads that share one row
        pkv.pkv_attention_expanded(out, q, k[:, :1].expand(4, 2, 64), k, r, s, s, 4)
    with pytest.raises(pkv.PagedKVError):
        pkv.pkv_attention_expanded(*ok, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert pkv.device_error() == 0
