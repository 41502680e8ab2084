"""Refusals of the device-table and sparse-attention entry points (CPU: nothing is
launched)."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


def _tables(lib, **kw):
    f = dict(block_table=1 << 21, free_list=1 << 20, free_count=1 << 20, max_seqs=8, max_blocks=4,
             num_blocks=32, block_size=16)
    f.update(kw)
    return lib.DeviceTablesDesc(*(f[n] for n, _ in lib.DeviceTablesDesc._fields_))


def _step(lib, t, n=2, tokens=2, ptr=None, width=4, **kw):
    a = dict(rows=None, cached=FAKE, new=None, count=None, tables=FAKE, ctx=FAKE, start=FAKE,
             slots=FAKE, pos=FAKE)
    a.update(kw)
    return lib.lib().pkv_tables_step(t if t is None else ctypes.byref(t), a["rows"], a["cached"],
                                     a["new"], n, tokens, a["count"], a["tables"], width,
                                     a["ctx"], a["start"], a["slots"], a["pos"], None)


def test_tables_step_refuses(lib):
    bad = lib.PKV_ERR_INVALID
    assert _step(lib, None) == bad
    for field in ("block_table", "free_list", "free_count"):
        assert _step(lib, _tables(lib, **{field: None})) == bad
        assert _step(lib, _tables(lib, **{field: (1 << 20) + 2})) == bad
    for field in ("max_seqs", "max_blocks", "num_blocks", "block_size"):
        assert _step(lib, _tables(lib, **{field: 0})) == bad
    t = _tables(lib)
    assert _step(lib, t, n=-1) == bad and _step(lib, t, tokens=-1) == bad
    assert _step(lib, t, width=0) == bad
    for name in ("cached", "ctx", "start", "slots"):
        assert _step(lib, t, **{name: None}) == bad, name
    for name in ("rows", "cached", "new", "count", "tables", "ctx", "start", "slots", "pos"):
        assert _step(lib, t, **{name: ODD}) == bad, name
    own = _tables(lib, block_table=(1 << 20) + 64)
    assert _step(lib, own, tables=ctypes.c_void_p((1 << 20) + 64)) == bad
    assert _step(lib, _tables(lib, max_seqs=262145)) == lib.PKV_ERR_UNSUPPORTED
    assert _step(lib, _tables(lib, num_blocks=1 << 30)) == lib.PKV_ERR_UNSUPPORTED
    assert _step(lib, _tables(lib, max_blocks=1 << 28)) == lib.PKV_ERR_UNSUPPORTED
    assert _step(lib, t, tokens=1 << 30) == lib.PKV_ERR_UNSUPPORTED
    assert _step(lib, t, width=1 << 30) == lib.PKV_ERR_UNSUPPORTED


def test_tables_release_refuses(lib):
    L, ref = lib.lib(), ctypes.byref
    bad = lib.PKV_ERR_INVALID
    t = _tables(lib)
    assert L.pkv_tables_release(None, None, FAKE, 1, None) == bad
    assert L.pkv_tables_release(ref(t), None, None, 1, None) == bad
    assert L.pkv_tables_release(ref(t), ODD, FAKE, 1, None) == bad
    assert L.pkv_tables_release(ref(t), None, FAKE, -1, None) == bad
    assert L.pkv_tables_release(ref(t), None, None, 0, None) == 0
    assert L.pkv_tables_release(ref(_tables(lib, max_blocks=0)), None, FAKE, 1, None) == bad


def _desc(lib, **kw):
    f = dict(dtype=lib.PKV_BF16, num_blocks=100, block_size=16, num_kv_heads=8, num_q_heads=32,
             head_dim=128)
    f.update(kw)
    return lib.CacheDesc(*(f[n] for n, _ in lib.CacheDesc._fields_))


UNSUPPORTED = [dict(dtype=2), dict(block_size=32), dict(head_dim=96), dict(num_q_heads=24)]


def _bounds(lib, d, n=2, tokens=2, width=4, **kw):
    a = dict(b=FAKE, e=FAKE, k=FAKE, t=FAKE, s=None, c=FAKE)
    a.update(kw)
    return lib.lib().pkv_block_bounds(a["b"], a["e"], a["k"], ctypes.byref(d), a["t"], width,
                                      a["s"], a["c"], n, tokens, None)


def _select(lib, d, n=2, tokens=2, width=4, max_ctx=64, top_k=4, sink=1, recent=1, ws=FAKE,
            ws_bytes=1 << 20, **kw):
    a = dict(o=FAKE, q=FAKE, b=FAKE, e=FAKE, t=FAKE, s=None, c=FAKE)
    a.update(kw)
    return lib.lib().pkv_select_blocks(a["o"], a["q"], a["b"], a["e"], ctypes.byref(d), a["t"],
                                       width, a["s"], a["c"], n, tokens, max_ctx, top_k, sink,
                                       recent, ws, ws_bytes, None)


def _attend(lib, d, n=2, tokens=2, width=4, top_k=4, scale=0.1, **kw):
    a = dict(o=FAKE, q=FAKE, k=FAKE, v=FAKE, t=FAKE, s=None, c=FAKE, l=FAKE)
    a.update(kw)
    return lib.lib().paged_attention_sparse(a["o"], a["q"], a["k"], a["v"], ctypes.byref(d),
                                            a["t"], width, a["s"], a["c"], a["l"], top_k, n,
                                            tokens, scale, None)


@pytest.mark.parametrize("call,ptrs", [(_bounds, "bektc"), (_select, "oqbetc"),
                                       (_attend, "oqkvtcl")])
def test_sparse_entry_points_refuse(lib, call, ptrs):
    bad = lib.PKV_ERR_INVALID
    d = _desc(lib)
    for kw in UNSUPPORTED:
        assert call(lib, _desc(lib, **kw)) == lib.PKV_ERR_UNSUPPORTED, kw
    assert call(lib, _desc(lib, num_q_heads=31)) == bad
    assert call(lib, d, n=-1) == bad and call(lib, d, tokens=-1) == bad
    assert call(lib, d, width=0) == bad
    assert call(lib, d, tokens=3) == bad             # more rows than sequences, no layout
    for name in ptrs:
        assert call(lib, d, **{name: None}) == bad, name
        if name != "e":                              # exponents are bytes
            assert call(lib, d, **{name: ODD}) == bad, name
    assert call(lib, d, s=ODD) == bad
    # nothing to do whatever the pointers hold
    none = {name: None for name in ptrs}
    assert call(lib, d, n=0, tokens=0, **none) == 0
    assert call(lib, d, n=2, tokens=0, s=FAKE, **none) == 0


def test_select_and_attend_scalars(lib):
    d, bad = _desc(lib), lib.PKV_ERR_INVALID
    assert _select(lib, d, top_k=0) == bad
    assert _select(lib, d, sink=-1) == bad and _select(lib, d, recent=0) == bad
    assert _select(lib, d, top_k=4, sink=3, recent=2) == bad
    assert _select(lib, d, max_ctx=0) == bad
    many = 1 << 28
    assert _select(lib, d, top_k=many) == lib.PKV_ERR_UNSUPPORTED
    assert _select(lib, d, n=many, tokens=many) == lib.PKV_ERR_UNSUPPORTED
    wide = _desc(lib, num_kv_heads=1 << 12, num_q_heads=1 << 12)
    assert _select(lib, wide, max_ctx=1 << 30) == lib.PKV_ERR_UNSUPPORTED
    assert _attend(lib, d, top_k=many) == lib.PKV_ERR_UNSUPPORTED
    assert _attend(lib, d, n=many, tokens=many) == lib.PKV_ERR_UNSUPPORTED
    assert _bounds(lib, d, n=many, tokens=many) == lib.PKV_ERR_UNSUPPORTED
    assert _select(lib, d, ws=None) == lib.PKV_ERR_WORKSPACE
    assert _select(lib, d, ws=ctypes.c_void_p((1 << 20) + 16)) == lib.PKV_ERR_WORKSPACE
    assert _select(lib, d, ws_bytes=16) == lib.PKV_ERR_WORKSPACE
    assert _attend(lib, d, top_k=0) == bad
    assert _attend(lib, d, scale=float("nan")) == bad
    assert _attend(lib, d, scale=float("inf")) == bad


def test_select_workspace_grows_with_rows_and_context(lib):
    d = _desc(lib)
    a = lib.select_workspace_bytes(d, 64, 32768)
    assert a >= 64 * 8 * 2048 * 4 and a % 256 == 0
    assert lib.select_workspace_bytes(d, 64, 4096) < a
    assert lib.select_workspace_bytes(d, 65, 32768) > a
    assert lib.select_workspace_bytes(_desc(lib, dtype=2), 64, 4096) == 0
    assert lib.select_workspace_bytes(d, -1, 4096) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        lib.DeviceTables(t, t[0], t[0, :1], 16)
    with pytest.raises(ValueError):
        lib.DeviceTables.create(4, 16, 2, 2, free_order=[0, 1], device="cpu")
    d = lib.CacheDesc(lib.PKV_F32, 4, 16, 1, 1, 64)
    q, k = torch.zeros(1, 1, 64), torch.zeros(4, 1, 16, 64)
    b, e = torch.zeros((4, 1, 2, 64), dtype=torch.int8), torch.zeros((4, 1), dtype=torch.int8)
    ctx, sel = torch.ones(1, dtype=torch.int32), torch.zeros((1, 1, 1), dtype=torch.int32)
    with pytest.raises(TypeError, match="bounds must be a contiguous CUDA"):
        lib.pkv_block_bounds(b, e, k, d, t[:1], ctx)
    with pytest.raises(TypeError, match="selected must be a contiguous CUDA"):
        lib.pkv_select_blocks(sel, q, b, e, d, t[:1], ctx, 16, 0, 1, ws=b)
    with pytest.raises(TypeError, match="out must be a contiguous CUDA"):
        lib.paged_attention_sparse(q, q, k, k, d, t[:1], ctx, sel)
    with pytest.raises(TypeError, match="must be a tensor"):
        lib.paged_attention_sparse(None, q, k, k, d, t[:1], ctx, sel)
    hot = lib._native()
    with pytest.raises(TypeError, match="arguments expected"):
        hot.attention_sparse(q)
