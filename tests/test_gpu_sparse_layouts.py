"""GPU: query layouts that do not fit their call, through the sparse entry points:
flagged, and no memory outside the outputs and the workspace touched."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import sparse  # noqa: E402
from tests.sparse_checks import (assert_attention, attention_bound, i32, tables_for,  # noqa: E402
                                 to_dev, values)

pytestmark = pytest.mark.gpu

BAD_LAYOUT = 5                                     # PKV_DEV_BAD_QUERY_LAYOUT


@pytest.fixture(scope="module")
def pkv(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lib.device_error(clear=True)
    return lib


def fenced(x, byte=0x5A, before=4096, behind=1 << 20):
    """A copy of tensor x in the middle of a buffer of `byte`, and a check that the
    bytes around it are still that."""
    n = x.numel() * x.element_size()
    buf = torch.full((before + n + behind,), byte, dtype=torch.uint8, device="cuda")
    y = buf[before:before + n].view(x.dtype).view(x.shape)
    y.copy_(x)

    def whole():
        return bool((buf[:before] == byte).all()) and bool((buf[before + n:] == byte).all())

    return y, whole


class Batch:
    """Tables, bounds, caches and query rows of a few sequences; every output and the
    workspace (of exactly the size asked for) lie between fences."""

    def __init__(self, pkv, dtype, hq, hkv, ctx, rows, top_k=4, d=64):
        self.pkv, self.dtype, self.ctx = pkv, dtype, ctx
        rng = np.random.default_rng(hq + 10 * hkv + rows)
        self.t, nb = tables_for(rng, ctx)
        self.k, self.v = (values(rng, (nb, hkv, 16, d), dtype) for _ in range(2))
        self.q = values(rng, (rows, hq, d), dtype)
        self.b = np.zeros((nb, hkv, 2, d), np.int8)
        self.e = np.zeros((nb, hkv), np.int8)
        sparse.update_bounds(self.b, self.e, self.k, self.t,
                             np.concatenate([[0], np.cumsum(ctx)]), ctx, dtype)
        self.kd, self.vd = to_dev(self.k, dtype), to_dev(self.v, dtype)
        self.desc = pkv.cache_desc(self.kd, hq)
        self.max_ctx, self.top_k = max(ctx), top_k
        self.qd, self.q_whole = fenced(to_dev(self.q, dtype), 0xFF)   # NaN behind the rows
        self.sel0 = torch.full((rows, hkv, top_k), -9, dtype=torch.int32, device="cuda")
        self.out0 = torch.full((rows, hq, d), 7.0, dtype=self.kd.dtype, device="cuda")
        self.lists = np.zeros((rows, hkv, top_k), np.int32)           # block 0, four times

    def bounds(self, start, tokens):
        """(what the call wrote, bounds then exponents, else 99)"""
        b, b_whole = fenced(torch.full(self.b.shape, 99, dtype=torch.int8, device="cuda"))
        e, e_whole = fenced(torch.full(self.e.shape, 99, dtype=torch.int8, device="cuda"))
        self.pkv.pkv_block_bounds(b, e, self.kd, self.desc, i32(self.t), i32(self.ctx),
                                  query_start_loc=i32(start), num_query_tokens=tokens)
        code = self.pkv.device_error()
        assert b_whole() and e_whole()
        return code, b.cpu().numpy(), e.cpu().numpy()

    def select(self, start, ws_byte=0x00):
        need = self.pkv.select_workspace_bytes(self.desc, self.q.shape[0], self.max_ctx)
        ws, ws_whole = fenced(torch.full((need,), ws_byte, dtype=torch.uint8, device="cuda"))
        sel, sel_whole = fenced(self.sel0)
        self.pkv.pkv_select_blocks(sel, self.qd, to_dev(self.b), to_dev(self.e), self.desc,
                                   i32(self.t), i32(self.ctx), self.max_ctx, 1, 1,
                                   query_start_loc=i32(start), ws=ws)
        code = self.pkv.device_error()
        assert ws_whole() and sel_whole() and self.q_whole()
        return code, sel.cpu().numpy()

    def attend(self, start):
        out, out_whole = fenced(self.out0)
        self.pkv.paged_attention_sparse(out, self.qd, self.kd, self.vd, self.desc, i32(self.t),
                                        i32(self.ctx), i32(self.lists), query_start_loc=i32(start))
        code = self.pkv.device_error()
        assert out_whole() and self.q_whole()
        return code, out


@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 2, 2), ("bf16", 4, 2), ("f32", 4, 1),
                                          ("f32", 8, 1)])
@pytest.mark.parametrize("rows,start,ctx", [
    (5, [0, 8], [700]),                            # the only sequence goes past the rows
    (5, [0, 1, 3, 12], [300, 700, 500]),           # the last one does
    (3, [0, 3, 4], [700, 400]),                    # a sequence wholly behind them
    (6, [0, 100, 6], [2000, 300]),                 # one that ends above the end of all
])
def test_layouts_past_the_rows_are_flagged(pkv, dtype, hq, hkv, rows, start, ctx):
    """Groups of query rows that share their reads end with the call's rows."""
    batch = Batch(pkv, dtype, hq, hkv, ctx, rows)
    past = start[-1] > rows                        # nothing at all is written
    code, b, e = batch.bounds(start, rows)
    assert code == BAD_LAYOUT
    if past:
        assert (b == 99).all() and (e == 99).all()
    code, sel = batch.select(start)
    assert code == BAD_LAYOUT
    if past:
        assert (sel == -9).all()
    code, out = batch.attend(start)
    assert code == BAD_LAYOUT
    if past:
        assert (out == 7.0).all()


@pytest.mark.parametrize("rows,start,ctx", [(8, [0, 5], [700]), (9, [0, 1, 1, 4], [300, 5, 500])])
def test_padded_layouts_stay_served(pkv, rows, start, ctx):
    batch = Batch(pkv, "bf16", 4, 2, ctx, rows)
    m = start[-1]
    code, b, e = batch.bounds(start, rows)
    ref_b, ref_e = np.full_like(batch.b, 99), np.full_like(batch.e, 99)
    sparse.update_bounds(ref_b, ref_e, batch.k, batch.t, start, ctx, "bf16")
    assert code == 0 and np.array_equal(b, ref_b) and np.array_equal(e, ref_e)
    code, sel = batch.select(start)
    ref = sparse.select(batch.q, batch.b, batch.e, batch.t, start, ctx, 16, 4, 1, 1, "bf16")
    assert code == 0 and np.array_equal(sel[:m], ref[:m]) and (sel[m:] == -9).all()
    code, out = batch.attend(start)
    assert code == 0 and (out[m:] == 7.0).all()
    args = (batch.q[:m], batch.k, batch.v, batch.t, start, ctx, batch.lists[:m], "bf16")
    ref = sparse.attention(*args)
    assert_attention(out[:m], ref, attention_bound(*args, ref))


@pytest.mark.parametrize("ws_byte", [0x00, 0xFF])
@pytest.mark.parametrize("dtype,hq,hkv", [("bf16", 2, 2), ("bf16", 4, 2), ("f32", 8, 1)])
@pytest.mark.parametrize("rows,start,ctx", [
    (8, [0, 5, 2, 8], [700, 900, 400]),            # every row belongs to a sequence all the same
    (8, [-3, 8], [700]),                           # rows that begin before the batch
    (8, [3, 8], [700]),                            # rows of no sequence in front
    (9, [0, 4, 4, 3, 9], [500, 20, 700, 640]),
    (12, [0, 9, 1, 12, 2, 12], [300, 1500, 2500, 700, 900]),
])
def test_layouts_out_of_order_are_flagged(pkv, dtype, hq, hkv, rows, start, ctx, ws_byte):
    """Whatever the workspace held before: rows whose group leads in another sequence
    find scores there that no warp wrote."""
    batch = Batch(pkv, dtype, hq, hkv, ctx, rows)
    assert batch.bounds(start, rows)[0] == BAD_LAYOUT
    code, sel = batch.select(start, ws_byte)
    assert code == BAD_LAYOUT
    assert ((sel == -9) | ((sel >= -1) & (sel < -(-max(ctx) // 16)))).all()
    assert batch.attend(start)[0] == BAD_LAYOUT


@pytest.mark.parametrize("blocks", [600, 2100, 9000])
def test_layouts_out_of_order_over_long_rows(pkv, blocks):
    """Every length of row that the lists are made for, over a workspace of ones."""
    batch = Batch(pkv, "bf16", 2, 2, [blocks * 16, 300, blocks * 16 - 5], 8, top_k=40)
    code, sel = batch.select([0, 5, 2, 8], 0xFF)
    assert code == BAD_LAYOUT and (sel < blocks).all()


def test_many_empty_sequences_are_looked_over(pkv):
    """More offsets than the kernels have threads, one of them out of order."""
    n, rows = 70000, 4
    rng = np.random.default_rng(3)
    ctx = np.ones(n, dtype=np.int64)
    ctx[n - 1] = 700
    t = np.full((n, 44), -1, dtype=np.int32)
    t[:, 0] = 0
    t[n - 1] = rng.permutation(44)
    kd = to_dev(values(rng, (44, 1, 16, 64), "f32"))
    desc = pkv.cache_desc(kd, 1)
    qd = to_dev(values(rng, (rows, 1, 64), "f32"))
    td, cd = i32(t), i32(ctx)
    bb = pkv.BlockBounds(44, 1, 64)
    sel = torch.full((rows, 1, 4), -9, dtype=torch.int32, device="cuda")
    for bad in (None, 1, n // 2, n - 2):
        start = np.zeros(n + 1, dtype=np.int64)
        start[n] = rows
        if bad is not None:
            start[bad] = 1
        sd = i32(start)
        want = 0 if bad is None else BAD_LAYOUT
        pkv.pkv_block_bounds(bb.bounds, bb.exps, kd, desc, td, cd, query_start_loc=sd,
                             num_query_tokens=rows)
        assert pkv.device_error() == want
        pkv.pkv_select_blocks(sel, qd, bb.bounds, bb.exps, desc, td, cd, 704, 1, 1,
                              query_start_loc=sd)
        assert pkv.device_error() == want
        pkv.paged_attention_sparse(torch.empty_like(qd), qd, kd, kd, desc, td, cd, sel.clamp(min=0),
                                   query_start_loc=sd)
        assert pkv.device_error() == want
