"""Chunk append, read back, chunk attention and windowed decode: what the host refuses before any launch (CPU)."""
import ctypes

import pytest
import torch

from bit_kv_cache_16_b200 import build, kvq

from test_abi import _fake_cache, _shape

BAD, ALIGN, WS, SHAPE = (kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_ALIGNMENT, kvq.KVQ_ERR_WORKSPACE, kvq.KVQ_ERR_SHAPE)


@pytest.fixture(scope="module")
def lib():
    build.build_libkvq()
    return kvq.load()


def call(lib, name, cache, **kw):
    """The entry point with aligned dummy arguments, some replaced."""
    args = {
        "kvq_append_chunk": dict(k=16, v=16, cls=None, cu=16, total_new=8, max_new=8, stream=None),
        "kvq_read_tokens": dict(start=16, cu=16, total=8, max_len=8, k=16, v=16, stream=None),
        "kvq_chunk_attention": dict(q=16, k=16, v=16, cu=16, total_new=8, max_new=8, scale=1.0, window=0, sinks=0,
                                    out=16, ws=16, ws_bytes=1 << 40, splits=0, max_len=8192, stream=None),
        "kvq_decode_attention_window": dict(q=16, out=16, lse=16, scale=1.0, window=64, sinks=4, ws=16,
                                            ws_bytes=1 << 40, splits=0, max_len=8192, stream=None),
    }[name]
    args.update(kw)
    return getattr(lib, name)(ctypes.byref(cache) if cache is not None else None, *args.values())


@pytest.mark.parametrize("name,kw,status", [
    ("kvq_append_chunk", dict(k=None), BAD), ("kvq_append_chunk", dict(v=None), BAD),
    ("kvq_append_chunk", dict(cu=None), BAD), ("kvq_append_chunk", dict(max_new=-1), BAD),
    ("kvq_append_chunk", dict(cls=16), BAD), ("kvq_append_chunk", dict(total_new=-1), BAD),
    ("kvq_read_tokens", dict(total=-1), BAD), ("kvq_append_chunk", dict(k=24), ALIGN),
    ("kvq_append_chunk", dict(cu=18), ALIGN),
    ("kvq_read_tokens", dict(cu=None), BAD), ("kvq_read_tokens", dict(max_len=-1), BAD),
    ("kvq_read_tokens", dict(k=None, v=None), BAD), ("kvq_read_tokens", dict(v=24), ALIGN),
    ("kvq_read_tokens", dict(start=18), ALIGN),
    ("kvq_chunk_attention", dict(q=None), BAD), ("kvq_chunk_attention", dict(k=None), BAD),
    ("kvq_chunk_attention", dict(out=None), BAD), ("kvq_chunk_attention", dict(cu=None), BAD),
    ("kvq_chunk_attention", dict(scale=float("nan")), BAD), ("kvq_chunk_attention", dict(window=-1), BAD),
    ("kvq_chunk_attention", dict(sinks=-1), BAD), ("kvq_chunk_attention", dict(splits=-1), BAD),
    ("kvq_chunk_attention", dict(splits=65536), BAD), ("kvq_chunk_attention", dict(total_new=-1), BAD),
    ("kvq_chunk_attention", dict(max_new=-1), BAD), ("kvq_chunk_attention", dict(max_len=-1), BAD),
    ("kvq_chunk_attention", dict(q=24), ALIGN), ("kvq_chunk_attention", dict(out=24), ALIGN),
    ("kvq_chunk_attention", dict(ws=24), ALIGN),
    ("kvq_decode_attention_window", dict(q=None), BAD), ("kvq_decode_attention_window", dict(out=None), BAD),
    ("kvq_decode_attention_window", dict(scale=float("nan")), BAD),
    ("kvq_decode_attention_window", dict(window=-1), BAD), ("kvq_decode_attention_window", dict(sinks=-1), BAD),
    ("kvq_decode_attention_window", dict(splits=-1), BAD), ("kvq_decode_attention_window", dict(max_len=-1), BAD),
    ("kvq_decode_attention_window", dict(lse=24), ALIGN), ("kvq_decode_attention_window", dict(out=24), ALIGN),
])
def test_refused_arguments(lib, name, kw, status):
    assert call(lib, name, _fake_cache(_shape()), **kw) == status


@pytest.mark.parametrize("name", ["kvq_append_chunk", "kvq_read_tokens", "kvq_chunk_attention",
                                  "kvq_decode_attention_window"])
def test_refused_caches(lib, name):
    assert call(lib, name, None) == BAD
    assert call(lib, name, _fake_cache(_shape(num_q_heads=30))) == SHAPE
    assert call(lib, name, _fake_cache(_shape(), v_meta=0)) == BAD
    assert call(lib, name, _fake_cache(_shape(), k_res=0x1008)) == ALIGN


def test_append_chunk_needs_the_classes_of_a_mixed_cache(lib):
    m = _fake_cache(_shape(format=6))
    assert call(lib, "kvq_append_chunk", m, cls=None) == BAD


def test_workspaces(lib):
    """More splits need more; one byte less than the stated size, or none at all, is refused."""
    c = _fake_cache(_shape())
    for rows, max_new, max_len, window, sinks in ((8, 1, 8192, 0, 0), (64, 8, 8192, 1024, 4), (1, 1, 1, 0, 0)):
        need = [lib.kvq_chunk_workspace_bytes(ctypes.byref(c), n, rows, max_new, max_len, window, sinks)
                for n in (1, 2, 5)]
        assert need[0] <= need[1] <= need[2]
        for n, bytes_ in zip((1, 2, 5), need):
            if bytes_:
                assert call(lib, "kvq_chunk_attention", c, total_new=rows, max_new=max_new, window=window,
                            sinks=sinks, splits=n, ws_bytes=bytes_ - 1) == WS
                assert call(lib, "kvq_chunk_attention", c, total_new=rows, max_new=max_new, window=window,
                            sinks=sinks, splits=n, ws=None) == BAD
    for n in (2, 5):
        bytes_ = lib.kvq_window_workspace_bytes(ctypes.byref(c), n, 8192, 1024, 4)
        if bytes_:
            assert call(lib, "kvq_decode_attention_window", c, splits=n, ws_bytes=bytes_ - 1) == WS
    assert lib.kvq_chunk_workspace_bytes(ctypes.byref(c), -1, 8, 1, 8192, 0, 0) == 0
    assert lib.kvq_window_workspace_bytes(ctypes.byref(c), 0, 8192, -1, 0) == 0
    assert lib.kvq_window_workspace_bytes(None, 0, 8192, 1, 0) == 0


def test_no_rows_no_launch(lib):
    """A chunk attention over no rows at all needs no device."""
    assert call(lib, "kvq_chunk_attention", _fake_cache(_shape()), q=None, k=None, v=None, out=None, total_new=0,
                max_new=0) == kvq.KVQ_OK


class _Stub(kvq.Cache):
    """A Cache around dummy pointers, for the checks that come before the library is called."""

    def __init__(self):
        self.shape = _shape()
        self.device = torch.device("cpu")
        self._index = -1
        self.desc = _fake_cache(self.shape)


def test_python_checks():
    c = _Stub()
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    cu = torch.zeros(9, dtype=torch.int32)
    k, q, out = bf(5, 8, 128), bf(5, 32, 128), bf(5, 32, 128)
    ws = torch.zeros(16, dtype=torch.uint8)
    for bad in (dict(k=k.float()), dict(k=bf(5, 4, 128)), dict(v=bf(4, 8, 128)), dict(cu=cu[:8]), dict(cu=cu.long()),
                dict(k=bf(8, 5, 128).transpose(0, 1)), dict(cls=torch.zeros(4, dtype=torch.uint8))):
        a = dict(k=k, v=k, cu=cu, cls=None)
        a.update(bad)
        with pytest.raises(ValueError):
            c.append_chunk(a["k"], a["v"], a["cu"], 5, token_class=a["cls"])
    for bad in (dict(start=cu), dict(k=bf(5, 8, 64)), dict(v=k.float()), dict(cu=cu[1:])):
        a = dict(start=cu[:8].contiguous(), cu=cu, k=k, v=k)
        a.update(bad)
        with pytest.raises(ValueError):
            c.read_tokens(a["start"], a["cu"], 5, a["k"], a["v"])
    for bad in (dict(q=q[:, :8]), dict(k=k[:4]), dict(out=out.float()), dict(ws=ws[::2]), dict(cu=cu.float()[:8])):
        a = dict(q=q, k=k, v=k, cu=cu, out=out, ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            c.chunk_attention(a["q"], a["k"], a["v"], a["cu"], 5, a["out"], 1.0, a["ws"], 0, 10)
    q1, o1, lse = bf(8, 32, 128), torch.zeros(8, 32, 128), torch.zeros(8, 32)
    for bad in (dict(q=q), dict(out=out), dict(lse=lse[:4]), dict(ws=ws[::2])):
        a = dict(q=q1, out=o1, lse=lse, ws=ws)
        a.update(bad)
        with pytest.raises(ValueError):
            c.decode_attention_window(a["q"], a["out"], 1.0, 4, 0, a["ws"], 0, 10, lse=a["lse"])
