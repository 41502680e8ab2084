"""Refusals of the latent-attention entry points (CPU: nothing is launched)."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)
HALF = ctypes.c_void_p((1 << 20) + 8)              # a multiple of 8, not of 16


def _desc(lib, **kw):
    f = dict(dtype=lib.PKV_BF16, num_blocks=100, block_size=16, latent_dim=512, rope_dim=64,
             num_q_heads=24)
    f.update(kw)
    return lib.LatentDesc(*(f[n] for n, _ in lib.LatentDesc._fields_))


def _append(lib, d, n=2, most=64, layout=0, eps=1e-6, latent_stride=576, k_stride=576,
            q_strides=(4608, 192), o_strides=(13824, 576), **kw):
    a = dict(x=FAKE, k=FAKE, w=FAKE, s=FAKE, p=FAKE, t=FAKE, c=FAKE, q=FAKE, o=FAKE)
    a.update(kw)
    return lib.lib().paged_latent_append(a["x"], latent_stride, a["k"], k_stride, a["w"], eps,
                                         a["s"], a["p"], a["t"], most, layout, n, a["c"], a["q"],
                                         *q_strides, a["o"], *o_strides, ctypes.byref(d), None)


def _copy(lib, d, n=2, **kw):
    a = dict(p=FAKE, c=FAKE)
    a.update(kw)
    return lib.lib().pkv_copy_blocks_latent(a["p"], n, a["c"], ctypes.byref(d), None)


def _gather(lib, d, n=2, keys=9, width=4, **kw):
    a = dict(x=FAKE, r=FAKE, c=FAKE, t=FAKE, s=FAKE)
    a.update(kw)
    return lib.lib().paged_latent_gather(a["x"], a["r"], a["c"], ctypes.byref(d), a["t"], width,
                                         a["s"], n, keys, None)


def _attend(lib, d, n=2, tokens=2, width=4, most=64, scale=0.1, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = dict(o=FAKE, q=FAKE, c=FAKE, t=FAKE, s=None, l=FAKE)
    a.update(kw)
    return lib.lib().paged_attention_latent(a["o"], a["q"], a["c"], ctypes.byref(d), a["t"], width,
                                            a["s"], a["l"], n, tokens, most, scale, ws, ws_bytes,
                                            None)


@pytest.mark.parametrize("call", [_append, _copy, _gather, _attend])
def test_descriptors_that_no_kernel_takes(lib, call):
    for kw in (dict(dtype=2), dict(block_size=32), dict(latent_dim=192), dict(latent_dim=640),
               dict(rope_dim=32), dict(num_q_heads=65537), dict(num_blocks=1 << 27)):
        assert call(lib, _desc(lib, **kw)) == lib.PKV_ERR_UNSUPPORTED, kw
    for name in ("num_blocks", "block_size", "latent_dim", "rope_dim", "num_q_heads"):
        assert call(lib, _desc(lib, **{name: 0})) == lib.PKV_ERR_INVALID, name


def test_append_refuses(lib):
    d, bad = _desc(lib), lib.PKV_ERR_INVALID
    assert _append(lib, d, n=-1) == bad and _append(lib, d, most=0) == bad
    assert _append(lib, d, layout=2) == lib.PKV_ERR_UNSUPPORTED
    for eps in (-1.0, float("nan"), float("inf")):
        assert _append(lib, d, eps=eps) == bad
    for name in "xksptc":
        assert _append(lib, d, **{name: None}) == bad, name
    for name in "xkwtcqo":
        assert _append(lib, d, **{name: HALF}) == bad, name
    for name in "sp":
        assert _append(lib, d, **{name: ODD}) == bad, name
    assert _append(lib, d, q=None) == bad and _append(lib, d, o=None) == bad
    assert _append(lib, d, latent_stride=577) == bad and _append(lib, d, k_stride=4) == bad
    assert _append(lib, d, q_strides=(4608, 196)) == bad
    assert _append(lib, d, o_strides=(13825, 576)) == bad
    assert _append(lib, _desc(lib, dtype=lib.PKV_F32), k_stride=578) == bad
    none = {name: None for name in "xkwsptcqo"}
    assert _append(lib, d, n=0, **none) == 0


def test_copy_refuses(lib):
    d, bad = _desc(lib), lib.PKV_ERR_INVALID
    assert _copy(lib, d, n=-1) == bad and _copy(lib, d, n=65536) == lib.PKV_ERR_UNSUPPORTED
    assert _copy(lib, d, p=None) == bad and _copy(lib, d, c=None) == bad
    assert _copy(lib, d, p=ODD) == bad and _copy(lib, d, c=HALF) == bad
    assert _copy(lib, d, n=0, p=None, c=None) == 0


def test_gather_refuses(lib):
    d, bad = _desc(lib), lib.PKV_ERR_INVALID
    assert _gather(lib, d, n=-1) == bad and _gather(lib, d, keys=-1) == bad
    assert _gather(lib, d, width=0) == bad
    for name in "xrcts":
        assert _gather(lib, d, **{name: None}) == bad, name
        assert _gather(lib, d, **{name: ODD}) == bad, name
    none = {name: None for name in "xrcts"}
    assert _gather(lib, d, n=0, **none) == 0 and _gather(lib, d, keys=0, **none) == 0


def test_attention_refuses(lib):
    d, bad = _desc(lib), lib.PKV_ERR_INVALID
    assert _attend(lib, d, n=-1) == bad and _attend(lib, d, tokens=-1) == bad
    assert _attend(lib, d, width=0) == bad and _attend(lib, d, most=0) == bad
    assert _attend(lib, d, tokens=3) == bad            # more rows than sequences, no layout
    for scale in (0.0, -0.1, float("nan"), float("inf")):
        assert _attend(lib, d, scale=scale) == bad, scale
    for name in "oqctl":
        assert _attend(lib, d, **{name: None}) == bad, name
        assert _attend(lib, d, **{name: ODD}) == bad, name
    assert _attend(lib, d, s=ODD) == bad
    assert _attend(lib, d, ws=None) == lib.PKV_ERR_WORKSPACE
    assert _attend(lib, d, ws=ctypes.c_void_p((1 << 20) + 16)) == lib.PKV_ERR_WORKSPACE
    assert _attend(lib, d, n=1 << 27, tokens=1 << 27) == lib.PKV_ERR_UNSUPPORTED
    none = {name: None for name in "oqctl"}
    assert _attend(lib, d, n=0, tokens=0, **none) == 0
    assert _attend(lib, d, tokens=0, s=FAKE, **none) == 0


def test_latent_workspace(lib):
    d = _desc(lib)
    assert lib.latent_workspace_bytes(d, 4, 4, 64) == lib.latent_workspace_bytes(d, 400, 900, 1 << 20)
    assert lib.latent_workspace_bytes(_desc(lib, latent_dim=128), 4, 4, 64) < \
        lib.latent_workspace_bytes(d, 4, 4, 64)
    assert lib.latent_workspace_bytes(_desc(lib, rope_dim=32), 4, 4, 64) == 0
    assert lib.latent_workspace_bytes(d, -1, 4, 64) == 0
    assert lib.latent_workspace_bytes(d, 4, 4, 0) == 0


def _edesc(lib, **kw):
    f = dict(dtype=lib.PKV_BF16, num_heads=6, head_dim=128, rope_dim=64, k_token_stride=1536,
             k_head_stride=256, v_token_stride=1536, v_head_stride=256)
    f.update(kw)
    return lib.ExpandedDesc(*(f[n] for n, _ in lib.ExpandedDesc._fields_))


def _expanded(lib, d, n=2, tokens=5, keys=9, most=4, scale=0.1, ws=FAKE, ws_bytes=1 << 40, **kw):
    a = dict(o=FAKE, q=FAKE, k=FAKE, v=FAKE, r=FAKE, s=FAKE, t=FAKE)
    a.update(kw)
    return lib.lib().pkv_attention_expanded(a["o"], a["q"], a["k"], a["v"], a["r"],
                                            ctypes.byref(d), a["s"], a["t"], n, tokens, keys, most,
                                            scale, ws, ws_bytes, None)


def test_expanded_refuses(lib):
    d, bad = _edesc(lib), lib.PKV_ERR_INVALID
    for kw in (dict(dtype=2), dict(head_dim=96), dict(rope_dim=32), dict(num_heads=65537)):
        assert _expanded(lib, _edesc(lib, **kw)) == lib.PKV_ERR_UNSUPPORTED, kw
    for name in ("num_heads", "head_dim", "rope_dim"):
        assert _expanded(lib, _edesc(lib, **{name: 0})) == bad, name
    for name in ("k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride"):
        for stride in (0, -256, 260):
            assert _expanded(lib, _edesc(lib, **{name: stride})) == bad, (name, stride)
    assert _expanded(lib, d, n=-1) == bad and _expanded(lib, d, tokens=-1) == bad
    assert _expanded(lib, d, keys=-1) == bad and _expanded(lib, d, most=-1) == bad
    for scale in (0.0, -0.1, float("nan"), float("inf")):
        assert _expanded(lib, d, scale=scale) == bad, scale
    for name in "oqkvrst":
        assert _expanded(lib, d, **{name: None}) == bad, name
        assert _expanded(lib, d, **{name: ODD}) == bad, name
    assert _expanded(lib, d, ws=None) == lib.PKV_ERR_WORKSPACE
    assert _expanded(lib, d, ws_bytes=16) == lib.PKV_ERR_WORKSPACE
    none = {name: None for name in "oqkvrst"}
    assert _expanded(lib, d, n=0, **none) == 0 and _expanded(lib, d, tokens=0, **none) == 0
    need = lib.lib().pkv_expanded_workspace_bytes
    assert need(ctypes.byref(d), 4, 100000) > need(ctypes.byref(d), 4, 1000) > 0
    assert need(ctypes.byref(_edesc(lib, head_dim=80)), 4, 1000) == 0


def test_binding_refuses(lib):
    cache = torch.zeros(4, 16, 192)
    d = lib.latent_desc(cache, 128, 2)
    assert (d.latent_dim, d.rope_dim, d.num_q_heads, d.dtype) == (128, 64, 2, lib.PKV_F32)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        lib.latent_desc(cache.half(), 128, 2)
    x, k, i, s = torch.zeros(1, 128), torch.zeros(1, 64), torch.zeros(1, dtype=torch.int32), \
        torch.zeros(1, dtype=torch.int64)
    with pytest.raises(TypeError, match="latent must be a contiguous CUDA"):
        lib.paged_latent_append(x, k, s, i, k, cache, d)
    with pytest.raises(TypeError, match="latent_out must be a contiguous CUDA"):
        lib.paged_latent_gather(x, k, cache, d, i[None], torch.zeros(2, dtype=torch.int32))
    q = torch.zeros(1, 2, 192)
    with pytest.raises(TypeError, match="out must be a contiguous CUDA"):
        lib.paged_attention_latent(q, q, cache, d, i[None], i, 16, 0.1, ws=x)
    with pytest.raises(TypeError, match="out must be a contiguous CUDA"):
        lib.pkv_attention_expanded(q, q, q, q, k, i, i, 1, ws=x)
    with pytest.raises(TypeError, match="must be a tensor"):
        lib.paged_attention_latent(None, q, cache, d, i[None], i, 16, 0.1, ws=x)
