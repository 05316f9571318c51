"""Python binding of libkvq (argument marshalling only).

Every function here forwards to the C entry point of the same name declared
in include/kvq.h; all work runs in the library's CUDA kernels.  PyTorch is
used for device memory and streams only.  If libkvq.so is missing the import
of the library fails loudly: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import LIB_PATH

KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_SHAPE = 2
KVQ_ERR_UNSUPPORTED = 3
KVQ_ERR_ALIGNMENT = 4
KVQ_ERR_WORKSPACE = 5
KVQ_ERR_CUDA = 6

KVQ_FORMAT_INT2 = 2
KVQ_FORMAT_INT4 = 4
KVQ_FORMAT_FP8_E4M3 = 8
KVQ_FORMAT_INT8 = 16
KVQ_FORMAT_MIXED = 6

KVQ_DEVERR_APPEND_FULL = 0x1
KVQ_DEVERR_PAGE_RANGE = 0x2
KVQ_DEVERR_PREFILL_LEN = 0x4
KVQ_DEVERR_WAIT_TIMEOUT = 0x8
KVQ_DEVERR_STATE = 0x10

REGIONS = ["k_codes", "k_meta", "v_codes", "v_meta", "k_res", "v_res", "seq_len", "n_quant",
           "page_table", "fp8_scale", "fp8_amax", "err_word", "group_bits", "window_class", "k_sparse", "v_sparse"]

EXPORTED = ["kvq_buffer_bytes", "kvq_quantize_prefill", "kvq_append_token", "kvq_flush_group", "kvq_append_flush",
            "kvq_quantize_prefill_mixed", "kvq_append_token_mixed", "kvq_append_flush_mixed",
            "kvq_append_chunk", "kvq_read_tokens", "kvq_chunk_attention", "kvq_chunk_workspace_bytes",
            "kvq_decode_attention_window", "kvq_window_workspace_bytes",
            "kvq_decode_attention", "kvq_decode_attention_lse", "kvq_merge_partials",
            "kvq_decode_attention_noalloc", "kvq_decode_workspace_bytes", "kvq_decode_default_splits",
            "kvq_read_error", "kvq_status_string", "kvq_version"]


class KvqShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("format", "batch", "num_q_heads", "num_kv_heads", "head_dim", "group", "residual",
                 "capacity", "page_size", "max_pages_per_seq", "num_pages")] + [("rope_theta", ctypes.c_float),
                                                                                ("sparse", ctypes.c_int32)]


class KvqCache(ctypes.Structure):
    _fields_ = [("shape", KvqShape)] + [(n, ctypes.c_void_p) for n in REGIONS]


class KvqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__("%s failed: %s (status %d)" % (fn, status_string(status), status))
        self.status = status


_lib = None


def load(path: Optional[str] = None):
    """Load libkvq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise ImportError("libkvq.so not found at %s; build it with bit_kv_cache_16_b200.build.build_libkvq()"
                          % path)
    lib = ctypes.CDLL(path)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    pc = ctypes.POINTER(KvqCache)
    sig = {
        "kvq_buffer_bytes": (i32, [ctypes.POINTER(KvqShape), i32, ctypes.POINTER(sz)]),
        "kvq_quantize_prefill": (i32, [pc, vp, vp, vp, i32, vp]),
        "kvq_append_token": (i32, [pc, vp, vp, vp]),
        "kvq_flush_group": (i32, [pc, vp]),
        "kvq_append_flush": (i32, [pc, vp, vp, vp]),
        "kvq_quantize_prefill_mixed": (i32, [pc, vp, vp, vp, vp, i32, vp]),
        "kvq_append_token_mixed": (i32, [pc, vp, vp, vp, vp]),
        "kvq_append_flush_mixed": (i32, [pc, vp, vp, vp, vp]),
        "kvq_append_chunk": (i32, [pc, vp, vp, vp, vp, i32, i32, vp]),
        "kvq_read_tokens": (i32, [pc, vp, vp, i32, i32, vp, vp, vp]),
        "kvq_chunk_attention": (i32, [pc, vp, vp, vp, vp, i32, i32, f32, i32, i32, vp, vp, sz, i32, i32, vp]),
        "kvq_chunk_workspace_bytes": (sz, [pc, i32, i32, i32, i32, i32, i32]),
        "kvq_decode_attention_window": (i32, [pc, vp, vp, vp, f32, i32, i32, vp, sz, i32, i32, vp]),
        "kvq_window_workspace_bytes": (sz, [pc, i32, i32, i32, i32]),
        "kvq_decode_attention": (i32, [pc, vp, vp, f32, vp, sz, i32, i32, vp]),
        "kvq_decode_attention_lse": (i32, [pc, vp, vp, vp, f32, vp, sz, i32, i32, vp]),
        "kvq_merge_partials": (i32, [vp, vp, i32, ctypes.c_int64, vp, vp, vp]),
        "kvq_decode_attention_noalloc": (i32, [pc, vp, vp, f32, i32, i32, vp]),
        "kvq_decode_workspace_bytes": (sz, [pc, i32, i32]),
        "kvq_decode_default_splits": (i32, [pc, i32]),
        "kvq_read_error": (i32, [pc, ctypes.POINTER(ctypes.c_uint32), vp]),
        "kvq_status_string": (ctypes.c_char_p, [i32]),
        "kvq_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _current_stream(index: int) -> int:
    """Handle of the device's current stream (the handle alone: a Stream object costs 3 us)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _stream(stream) -> ctypes.c_void_p:
    if type(stream) is int:
        return ctypes.c_void_p(stream)
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    return ctypes.c_void_p(t.data_ptr())


def _addr(t):
    """Address for a pointer argument (ctypes takes the number; None is NULL)."""
    return None if t is None else t if isinstance(t, int) else t.data_ptr()


def _check(fn: str, status: int):
    if status != KVQ_OK:
        raise KvqError(fn, status)


# --------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# --------------------------------------------------------------------------

def status_string(status: int) -> str:
    return load().kvq_status_string(status).decode()


def kvq_status_string(status: int) -> str:
    return status_string(status)


def kvq_version() -> str:
    return load().kvq_version().decode()


def kvq_buffer_bytes(shape: KvqShape, region: int) -> int:
    n = ctypes.c_size_t(0)
    _check("kvq_buffer_bytes", load().kvq_buffer_bytes(ctypes.byref(shape), region, ctypes.byref(n)))
    return n.value


def kvq_quantize_prefill(cache: KvqCache, k, v, cu_seqlens, max_len: int, stream=None):
    _check("kvq_quantize_prefill", load().kvq_quantize_prefill(ctypes.byref(cache), _ptr(k), _ptr(v),
                                                               _ptr(cu_seqlens), int(max_len), _stream(stream)))


def kvq_append_token(cache: KvqCache, k_new, v_new, stream=None):
    _check("kvq_append_token", load().kvq_append_token(ctypes.byref(cache), _ptr(k_new), _ptr(v_new),
                                                       _stream(stream)))


def kvq_flush_group(cache: KvqCache, stream=None):
    _check("kvq_flush_group", load().kvq_flush_group(ctypes.byref(cache), _stream(stream)))


def kvq_append_flush(cache: KvqCache, k_new, v_new, stream=None):
    _check("kvq_append_flush", load().kvq_append_flush(ctypes.byref(cache), _ptr(k_new), _ptr(v_new),
                                                       _stream(stream)))


def kvq_quantize_prefill_mixed(cache: KvqCache, k, v, token_class, cu_seqlens, max_len: int, stream=None):
    """Prefill of a MIXED cache: token_class uint8 [T_total] (2 or 4) on the device."""
    _check("kvq_quantize_prefill_mixed",
           load().kvq_quantize_prefill_mixed(ctypes.byref(cache), _ptr(k), _ptr(v), _ptr(token_class),
                                             _ptr(cu_seqlens), int(max_len), _stream(stream)))


def kvq_append_token_mixed(cache: KvqCache, k_new, v_new, token_class, stream=None):
    """Append to a MIXED cache: token_class uint8 [B] (2 or 4) on the device."""
    _check("kvq_append_token_mixed", load().kvq_append_token_mixed(ctypes.byref(cache), _ptr(k_new), _ptr(v_new),
                                                                   _ptr(token_class), _stream(stream)))


def kvq_append_flush_mixed(cache: KvqCache, k_new, v_new, token_class, stream=None):
    _check("kvq_append_flush_mixed", load().kvq_append_flush_mixed(ctypes.byref(cache), _ptr(k_new), _ptr(v_new),
                                                                   _ptr(token_class), _stream(stream)))


def kvq_append_chunk(cache: KvqCache, k_new, v_new, token_class, cu_seqlens, total_new: int, max_new: int,
                     stream=None):
    """Append a ragged chunk of new tokens (token_class: MIXED only, else None)."""
    _check("kvq_append_chunk",
           load().kvq_append_chunk(ctypes.byref(cache), _addr(k_new), _addr(v_new), _addr(token_class),
                                   _addr(cu_seqlens), int(total_new), int(max_new), _stream(stream)))


def kvq_read_tokens(cache: KvqCache, start, cu_seqlens, total: int, max_len: int, k_out, v_out, stream=None):
    """Token ranges of the cache as bf16 rows (start None: from token 0; k_out or v_out None: not read)."""
    _check("kvq_read_tokens",
           load().kvq_read_tokens(ctypes.byref(cache), _addr(start), _addr(cu_seqlens), int(total), int(max_len),
                                  _addr(k_out), _addr(v_out), _stream(stream)))


def kvq_chunk_attention(cache: KvqCache, q, k_new, v_new, cu_seqlens, total_new: int, max_new: int,
                        softmax_scale: float, window: int, sinks: int, out, workspace, ws_bytes: int,
                        num_splits: int, max_len: int, stream=None):
    """A chunk of new tokens attends to the cache and, causally, to itself."""
    _check("kvq_chunk_attention",
           load().kvq_chunk_attention(ctypes.byref(cache), _addr(q), _addr(k_new), _addr(v_new), _addr(cu_seqlens),
                                      int(total_new), int(max_new), float(softmax_scale), int(window), int(sinks),
                                      _addr(out), _addr(workspace), int(ws_bytes), int(num_splits), int(max_len),
                                      _stream(stream)))


def kvq_chunk_workspace_bytes(cache: KvqCache, num_splits: int, total_new: int, max_new: int, max_len: int,
                              window: int = 0, sinks: int = 0) -> int:
    return int(load().kvq_chunk_workspace_bytes(ctypes.byref(cache), int(num_splits), int(total_new), int(max_new),
                                                int(max_len), int(window), int(sinks)))


def kvq_decode_attention_window(cache: KvqCache, q, out, lse, softmax_scale: float, window: int, sinks: int,
                                workspace, ws_bytes: int, num_splits: int, max_len: int, stream=None):
    """Decode over the last `window` tokens and the first `sinks` (lse None: not written)."""
    _check("kvq_decode_attention_window",
           load().kvq_decode_attention_window(ctypes.byref(cache), _addr(q), _addr(out), _addr(lse),
                                              float(softmax_scale), int(window), int(sinks), _addr(workspace),
                                              int(ws_bytes), int(num_splits), int(max_len), _stream(stream)))


def kvq_window_workspace_bytes(cache: KvqCache, num_splits: int, max_len: int, window: int, sinks: int = 0) -> int:
    return int(load().kvq_window_workspace_bytes(ctypes.byref(cache), int(num_splits), int(max_len), int(window),
                                                 int(sinks)))


def kvq_decode_workspace_bytes(cache: KvqCache, num_splits: int, max_len: int) -> int:
    return int(load().kvq_decode_workspace_bytes(ctypes.byref(cache), int(num_splits), int(max_len)))


def kvq_decode_default_splits(cache: KvqCache, max_len: int) -> int:
    return int(load().kvq_decode_default_splits(ctypes.byref(cache), int(max_len)))


def kvq_decode_attention(cache: KvqCache, q, out, softmax_scale: float, workspace, ws_bytes: int,
                         num_splits: int, max_len: int, stream=None):
    _check("kvq_decode_attention",
           load().kvq_decode_attention(ctypes.byref(cache), _ptr(q), _ptr(out), float(softmax_scale),
                                       _ptr(workspace), int(ws_bytes), int(num_splits), int(max_len),
                                       _stream(stream)))


def kvq_decode_attention_lse(cache: KvqCache, q, out, lse, softmax_scale: float, workspace, ws_bytes: int,
                             num_splits: int, max_len: int, stream=None):
    """kvq_decode_attention that also writes each row's ln-sum-exp into
    `lse` (float [B][H_q])."""
    _check("kvq_decode_attention_lse",
           load().kvq_decode_attention_lse(ctypes.byref(cache), _ptr(q), _ptr(out), _ptr(lse), float(softmax_scale),
                                           _ptr(workspace), int(ws_bytes), int(num_splits), int(max_len),
                                           _stream(stream)))


def kvq_merge_partials(outs, lses, parts: int, rows: int, out, lse_out=None, stream=None):
    """Merge `parts` attentions of the same rows over disjoint token sets:
    outs float [parts][rows][128], lses float [parts][rows] -> out [rows][128]
    (and the merged ln-sum-exp into lse_out [rows] when given)."""
    _check("kvq_merge_partials",
           load().kvq_merge_partials(_ptr(outs), _ptr(lses), int(parts), int(rows), _ptr(out), _ptr(lse_out),
                                     _stream(stream)))


def kvq_decode_attention_noalloc(cache: KvqCache, q, out, softmax_scale: float, num_splits: int, max_len: int,
                                 stream=None):
    """Decode without a workspace: the split partials use the library's fixed
    device array (see include/kvq.h for its size and sharing rules)."""
    _check("kvq_decode_attention_noalloc",
           load().kvq_decode_attention_noalloc(ctypes.byref(cache), _ptr(q), _ptr(out), float(softmax_scale),
                                               int(num_splits), int(max_len), _stream(stream)))


def kvq_read_error(cache: KvqCache, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check("kvq_read_error", load().kvq_read_error(ctypes.byref(cache), ctypes.byref(v), _stream(stream)))
    return v.value


# --------------------------------------------------------------------------
# A cache whose buffers are torch device tensors
# --------------------------------------------------------------------------

# accepted types: bf16 rows may come as their bit patterns
_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_INT32, _UINT8, _FLOAT = (torch.int32,), (torch.uint8,), (torch.float32,)


class Cache:
    """Allocates every region of a cache (torch uint8 tensors on `device`)
    and keeps the C descriptor pointing at them."""

    def __init__(self, fmt: int, batch: int, num_q_heads: int, num_kv_heads: int, capacity: int,
                 group: int = 32, residual: int = 128, page_size: int = 0, max_pages_per_seq: int = 0,
                 num_pages: int = 0, head_dim: int = 128, device="cuda", rope_theta: float = 0.0,
                 sparse: bool = False):
        load()
        self.shape = KvqShape(fmt, batch, num_q_heads, num_kv_heads, head_dim, group, residual, capacity,
                              page_size, max_pages_per_seq, num_pages, float(rope_theta), int(sparse))
        self.device = torch.device(device)
        self.buffers = {}
        # seq_len and n_quant side by side (each 16-byte aligned), so that reset() is one launch
        n = max(kvq_buffer_bytes(self.shape, REGIONS.index("seq_len")), 16)
        self._counters = torch.zeros(2, (n + 15) // 16 * 16, dtype=torch.uint8, device=self.device)
        for i, name in enumerate(REGIONS):
            if name in ("seq_len", "n_quant"):
                self.buffers[name] = self._counters[0 if name == "seq_len" else 1, :n]
                continue
            n_bytes = kvq_buffer_bytes(self.shape, i)
            # torch's caching allocator hands out 256-byte aligned blocks
            t = torch.zeros(max(n_bytes, 16), dtype=torch.uint8, device=self.device) if n_bytes else None
            self.buffers[name] = t
        self._index = self._counters.get_device()
        self.desc = KvqCache(self.shape, *[self.buffers[n].data_ptr() if self.buffers[n] is not None else None
                                           for n in REGIONS])

    @property
    def fmt(self) -> int:
        return self.shape.format

    def region(self, name: str) -> torch.Tensor:
        return self.buffers[name]

    def seq_len(self) -> torch.Tensor:
        return self.buffers["seq_len"].view(torch.int32)

    def n_quant(self) -> torch.Tensor:
        return self.buffers["n_quant"].view(torch.int32)

    def set_page_table(self, table: torch.Tensor):
        t = self.buffers["page_table"].view(torch.int32).view(self.shape.batch, self.shape.max_pages_per_seq)
        t.copy_(table.to(torch.int32))

    def clear_error(self):
        self.buffers["err_word"].zero_()

    def error(self, stream=None) -> int:
        return kvq_read_error(self.desc, stream)

    def quantize_prefill(self, k, v, cu_seqlens, max_len: int, stream=None):
        kvq_quantize_prefill(self.desc, k, v, cu_seqlens, max_len, stream)

    def append_token(self, k_new, v_new, stream=None):
        kvq_append_token(self.desc, k_new, v_new, stream)

    def flush_group(self, stream=None):
        kvq_flush_group(self.desc, stream)

    def append_flush(self, k_new, v_new, stream=None):
        kvq_append_flush(self.desc, k_new, v_new, stream)

    def quantize_prefill_mixed(self, k, v, token_class, cu_seqlens, max_len: int, stream=None):
        kvq_quantize_prefill_mixed(self.desc, k, v, token_class, cu_seqlens, max_len, stream)

    def append_token_mixed(self, k_new, v_new, token_class, stream=None):
        kvq_append_token_mixed(self.desc, k_new, v_new, token_class, stream)

    def append_flush_mixed(self, k_new, v_new, token_class, stream=None):
        kvq_append_flush_mixed(self.desc, k_new, v_new, token_class, stream)

    # The calls below check their tensors (device, type, layout and shape) and
    # run on the cache's device, whatever the current one is.

    def _need(self, name: str, t, rows, tail, dtypes):
        """t is a contiguous tensor [rows, *tail] (rows None: any number) of one of these types on the cache's device."""
        shape = t.shape
        if (t.dtype in dtypes and shape[1:] == tail and (rows is None or shape[0] == rows) and
                len(shape) == 1 + len(tail) and t.get_device() == self._index and t.is_contiguous()):
            return
        if t.get_device() != self._index:
            raise ValueError("%s is on %s, the cache on %s" % (name, t.device, self.device))
        if t.dtype not in dtypes:
            raise ValueError("%s is %s, not %s" % (name, t.dtype, dtypes[0]))
        if len(shape) == 1 + len(tail) and shape[1:] == tail and (rows is None or shape[0] == rows):
            raise ValueError("%s is not contiguous" % name)
        raise ValueError("%s has shape %s, not %s" % (name, tuple(shape), ("*" if rows is None else rows,) + tail))

    def _bytes_of(self, workspace) -> int:
        """Bytes of a workspace tensor (contiguous, on the cache's device) or 0 for None."""
        if workspace is None:
            return 0
        if workspace.get_device() != self._index or not workspace.is_contiguous():
            raise ValueError("workspace is on %s or not contiguous (the cache is on %s)" % (workspace.device, self.device))
        return workspace.numel() * workspace.element_size()

    def _call(self, fn, stream, *args):
        """fn(descriptor, *args, stream) with the cache's device current, on its current stream unless one is given."""
        if stream is None:
            stream = _current_stream(self._index)
        if torch.cuda.current_device() == self._index:
            return fn(self.desc, *args, stream)
        with torch.cuda.device(self._index):
            return fn(self.desc, *args, stream)

    def reset(self, stream=None):
        """Empty the cache: every sequence has no token (the FP8 scales stay)."""
        if stream is None:
            self._counters.zero_()
            return
        handle = _stream(stream).value or 0
        # (no ExternalStream for the default stream's handle: torch takes 0 for "none given")
        s = torch.cuda.ExternalStream(handle, self._index) if handle else torch.cuda.default_stream(self._index)
        with torch.cuda.stream(s):
            self._counters.zero_()

    def append_chunk(self, k_new, v_new, cu_seqlens, max_new: int, token_class=None, stream=None):
        """Append a ragged chunk: k_new, v_new bf16 [T, H_kv, 128], cu_seqlens int32 [B + 1]; token_class uint8 [T] for a
        MIXED cache."""
        s = self.shape
        tail = (s.num_kv_heads, 128)
        self._need("k_new", k_new, None, tail, _BF16)
        self._need("v_new", v_new, k_new.shape[0], tail, _BF16)
        self._need("cu_seqlens", cu_seqlens, s.batch + 1, (), _INT32)
        if token_class is not None:
            self._need("token_class", token_class, k_new.shape[0], (), _UINT8)
        self._call(kvq_append_chunk, stream, k_new, v_new, token_class, cu_seqlens, k_new.shape[0], max_new)

    def read_tokens(self, start, cu_seqlens, max_len: int, k_out, v_out, stream=None):
        """Tokens [start, start + length) of every sequence as bf16 rows [T, H_kv, 128] (start None: 0; either output
        may be None)."""
        s = self.shape
        if start is not None:
            self._need("start", start, s.batch, (), _INT32)
        self._need("cu_seqlens", cu_seqlens, s.batch + 1, (), _INT32)
        rows = None
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is not None:
                self._need(name, t, rows, (s.num_kv_heads, 128), _BF16)
                rows = t.shape[0]
        self._call(kvq_read_tokens, stream, start, cu_seqlens, 0 if rows is None else rows, max_len, k_out, v_out)

    def chunk_workspace_bytes(self, num_splits: int, total_new: int, max_new: int, max_len: int, window: int = 0,
                              sinks: int = 0) -> int:
        return kvq_chunk_workspace_bytes(self.desc, num_splits, total_new, max_new, max_len, window, sinks)

    def chunk_attention(self, q, k_new, v_new, cu_seqlens, max_new: int, out, softmax_scale: float, workspace,
                        num_splits: int, max_len: int, window: int = 0, sinks: int = 0, stream=None):
        """out bf16 [T, H_q, 128]: the chunk's queries q over the cached tokens and, causally, over k_new, v_new."""
        s = self.shape
        rows = q.shape[0]
        self._need("q", q, None, (s.num_q_heads, 128), _BF16)
        self._need("k_new", k_new, rows, (s.num_kv_heads, 128), _BF16)
        self._need("v_new", v_new, rows, (s.num_kv_heads, 128), _BF16)
        self._need("out", out, rows, (s.num_q_heads, 128), _BF16)
        self._need("cu_seqlens", cu_seqlens, s.batch + 1, (), _INT32)
        self._call(kvq_chunk_attention, stream, q, k_new, v_new, cu_seqlens, rows, max_new, softmax_scale, window, sinks,
                   out, workspace, self._bytes_of(workspace), num_splits, max_len)

    def window_workspace_bytes(self, num_splits: int, max_len: int, window: int, sinks: int = 0) -> int:
        return kvq_window_workspace_bytes(self.desc, num_splits, max_len, window, sinks)

    def decode_attention_window(self, q, out, softmax_scale: float, window: int, sinks: int, workspace,
                                num_splits: int, max_len: int, lse=None, stream=None):
        """out float [B, H_q, 128]: one query per sequence over its last `window` tokens and its first `sinks`."""
        s = self.shape
        self._need("q", q, s.batch, (s.num_q_heads, 128), _BF16)
        self._need("out", out, s.batch, (s.num_q_heads, 128), _FLOAT)
        if lse is not None:
            self._need("lse", lse, s.batch, (s.num_q_heads,), _FLOAT)
        self._call(kvq_decode_attention_window, stream, q, out, lse, softmax_scale, window, sinks, workspace,
                   self._bytes_of(workspace), num_splits, max_len)

    def workspace_bytes(self, num_splits: int, max_len: int) -> int:
        return kvq_decode_workspace_bytes(self.desc, num_splits, max_len)

    def decode_attention(self, q, out, softmax_scale: float, workspace, num_splits: int, max_len: int,
                         stream=None):
        kvq_decode_attention(self.desc, q, out, softmax_scale, workspace, workspace.numel() * workspace.element_size(),
                             num_splits, max_len, stream)

    def decode_attention_lse(self, q, out, lse, softmax_scale: float, workspace, num_splits: int, max_len: int,
                             stream=None):
        kvq_decode_attention_lse(self.desc, q, out, lse, softmax_scale, workspace,
                                 workspace.numel() * workspace.element_size(), num_splits, max_len, stream)
