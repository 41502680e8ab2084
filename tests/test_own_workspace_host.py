"""Calls that take their own workspace take it on the stream that they run on (CPU:
the streams, the tensors and the native calls are stand-ins, nothing is launched)."""

import contextlib

import pytest
import torch

from tests.test_abi_host import _FakeStream, _FakeTensor


@pytest.fixture
def taken(lib, monkeypatch):
    """[(stream the workspace was taken on, or None for the current one, its bytes)]"""
    on, got = [None], []

    @contextlib.contextmanager
    def under(stream):
        on.append(stream)
        yield
        on.pop()

    def workspace(nbytes, device=None):
        got.append((on[-1], nbytes))
        return _FakeTensor(0, torch.uint8, (nbytes,))

    class Native:
        @staticmethod
        def select_blocks(*args):
            return 0

    class Library:
        def __getattr__(self, name):
            return lambda *args: 4096 if name.endswith("_bytes") else 0

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _FakeStream(0))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(lib, "workspace", workspace)
    monkeypatch.setattr(lib, "_native", Native)
    monkeypatch.setattr(lib, "lib", Library)
    monkeypatch.setattr(_FakeTensor, "record_stream", lambda self, stream: None, raising=False)
    return got


def _select(lib, **kw):
    i32, i8, bf = torch.int32, torch.int8, torch.bfloat16
    desc = lib.CacheDesc(lib.PKV_BF16, 64, 16, 8, 32, 128)
    lib.pkv_select_blocks(_FakeTensor(0, i32, (4, 8, 5)), _FakeTensor(0, bf, (4, 32, 128)),
                          _FakeTensor(0, i8, (64, 8, 2, 128)), _FakeTensor(0, i8, (64, 8)), desc,
                          _FakeTensor(0, i32, (4, 8)), _FakeTensor(0, i32, (4,)), 100, 1, 1, **kw)


def _dense(lib):
    i32, bf = torch.int32, torch.bfloat16
    cache = _FakeTensor(0, bf, (64, 8, 16, 128))
    row = _FakeTensor(0, bf, (4, 32, 128))
    return dict(out=row, q=row, k_cache=cache, v_cache=cache,
                desc=lib.CacheDesc(lib.PKV_BF16, 64, 16, 8, 32, 128),
                block_tables=_FakeTensor(0, i32, (4, 8)), context_lens=_FakeTensor(0, i32, (4,)),
                max_context_len=100)


def _decode(lib, **kw):
    lib.paged_attention_decode(**_dense(lib), **kw)


def _varlen(lib, **kw):
    lib.paged_attention_varlen(**_dense(lib), query_start_loc=_FakeTensor(0, torch.int32, (5,)),
                               max_query_len=1, **kw)


def _decode_int8(lib, **kw):
    a = _dense(lib)
    cache = type("Cache", (), {})()
    cache.desc = lib.CacheDesc(lib.PKV_INT8, 64, 16, 8, 32, 128)
    cache.kv_pool = _FakeTensor(0, torch.uint8, (64, 8, 2, lib.int8_tile_bytes(128)))
    lib.paged_attention_decode_int8(a["out"], a["q"], cache, a["block_tables"], a["context_lens"],
                                    100, **kw)


CALLS = [_select, _decode, _varlen, _decode_int8]


@pytest.mark.parametrize("call", CALLS)
def test_own_workspaces_belong_to_the_call_s_stream(lib, taken, call):
    side = _FakeStream(0)
    call(lib, stream=side)
    call(lib)
    call(lib, stream=side, ws=_FakeTensor(0, torch.uint8, (1 << 20,)))
    assert [s for s, _ in taken] == [side, None]


@pytest.mark.parametrize("call", CALLS)
def test_streams_of_another_device_are_refused_before_a_workspace_is_taken(lib, taken, call):
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(lib, stream=_FakeStream(1))
    assert not taken
