"""ctypes binding of ``libgemma_attn.so`` -- argument marshalling only.

Every function carries the name of the C entry point it calls (declared in
``include/gemma_attn.h``). Tensors are torch CUDA tensors; their device
pointers, the shapes read off them and the current CUDA stream are passed
through unchanged. There is no fallback: if the shared library is missing
the import fails.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgemma_attn.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        "libgemma_attn.so is not built (run `python -m hybrid_local_global_b200.build`); "
        "there is no fallback implementation")
_lib = ctypes.CDLL(_LIB_PATH)
LIB_PATH = _LIB_PATH

GEMMA_OK = 0
GEMMA_ERR_INVALID_ARG = 1
GEMMA_ERR_UNSUPPORTED = 2
GEMMA_ERR_SHARE_MISMATCH = 3
GEMMA_ERR_CAPACITY = 4
GEMMA_ERR_CUDA = 5
GEMMA_ERR_DEVICE_TIMEOUT = 6
GEMMA_ERR_DEVICE_RANGE = 7
GEMMA_F_SHARED = 1
GEMMA_F_KEQV = 2  # K = V on a global layer: no v_new, values read from the key cache
GEMMA_F_KV_INT8 = 4  # int8 KV cache (Int8KVCache buffers); added automatically for those
GEMMA_F_SOURCE_WINDOW = 8  # shared local layer after cached tokens: attend to the source call's window

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t


class gemma_kv_desc(ctypes.Structure):
    _fields_ = [("k_cache", _P), ("v_cache", _P), ("layer", _I), ("cache_cap", _I),
                ("window", _I), ("n_kv_heads", _I), ("head_dim", _I), ("rope_frac", _F),
                ("rope_theta", _F), ("shared_from", _I), ("k_eq_v", _I), ("kv_int8", _I)]


def _sig(name, restype, argtypes):
    f = getattr(_lib, name)
    f.restype = restype
    f.argtypes = argtypes
    return f


_prefill_ws = _sig("gemma_attn_prefill_workspace_size", _SZ, [_I, _I, _I, _I, _I, _I])
_prefill_ws_cached = _sig("gemma_attn_prefill_workspace_size_cached", _SZ,
                          [_I, _I, _I, _I, _I, _I, _I, ctypes.c_uint])
_prefill = _sig("gemma_attn_prefill", _I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                           _F, _F, _F, _P, _P, _P, _SZ, ctypes.c_uint, _P])
_decode_ws = _sig("gemma_attn_decode_workspace_size", _SZ, [_I, _I, _I, _I, _I, _I])
_decode = _sig("gemma_attn_decode", _I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I,
                                         _F, _F, _F, _P, _P, _SZ, ctypes.c_uint, _P])
_bind = _sig("gemma_kv_share_bind", _I, [ctypes.POINTER(gemma_kv_desc), ctypes.POINTER(gemma_kv_desc)])
_sched = _sig("gemma_layer_schedule", _I, [_I, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)])
_ranges = _sig("gemma_attn_visible_ranges", _I, [_P, _I, _I, _I, _P, _P])
_sync = _sig("gemma_attn_sync_status", _I, [_P])
_last = _sig("gemma_last_error", ctypes.c_char_p, [])
_wait = _sig("gemma_attn_set_wait_limit", _I, [ctypes.c_longlong])
_drop = _sig("gemma_attn_debug_drop_next_copy", _I, [_I])
_kv_bytes = _sig("gemma_kv_cache_bytes", _SZ, [_I, _I, _I, _I, ctypes.c_uint])
_prefill_paged = _sig("gemma_attn_prefill_paged", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _I,
                                                       _I, _F, _F, _F, _P, _P, _P, _SZ, ctypes.c_uint, _P])
_decode_paged = _sig("gemma_attn_decode_paged", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _I, _I,
                                                     _F, _F, _F, _P, _P, _SZ, ctypes.c_uint, _P])
_kv_codes = _sig("gemma_kv_codes_bytes", _SZ, [_I, _I, _I, _I])
_multi_ws = _sig("gemma_attn_decode_multi_workspace_size", _SZ, [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_uint])
_multi = _sig("gemma_attn_decode_multi", _I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I,
                                              _F, _F, _F, _P, _P, _SZ, ctypes.c_uint, _P])
_multi_paged = _sig("gemma_attn_decode_multi_paged", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _I,
                                                          _I, _I, _F, _F, _F, _P, _P, _SZ, ctypes.c_uint, _P])

EXPORTED = ["gemma_attn_prefill_workspace_size", "gemma_attn_prefill",
            "gemma_attn_decode_workspace_size", "gemma_attn_decode", "gemma_kv_share_bind",
            "gemma_layer_schedule", "gemma_attn_visible_ranges", "gemma_attn_sync_status",
            "gemma_last_error", "gemma_attn_set_wait_limit", "gemma_attn_debug_drop_next_copy",
            "gemma_kv_cache_bytes", "gemma_kv_codes_bytes", "gemma_attn_prefill_paged",
            "gemma_attn_decode_paged", "gemma_attn_prefill_workspace_size_cached"]


class GemmaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("gemma_attn error %d: %s" % (code, msg))
        self.code = code


def _check(rc: int) -> int:
    if rc != GEMMA_OK:
        raise GemmaError(rc, gemma_last_error())
    return rc


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def gemma_kv_cache_bytes(batch, n_kv_heads, cache_cap, head_dim, flags=0) -> int:
    return int(_kv_bytes(batch, n_kv_heads, cache_cap, head_dim, flags))


def gemma_kv_codes_bytes(batch, n_kv_heads, cache_cap, head_dim) -> int:
    return int(_kv_codes(batch, n_kv_heads, cache_cap, head_dim))


class Int8KVCache:
    """One layer's int8 K (or V) cache buffer (GEMMA_F_KV_INT8 layout):
    ``codes`` uint8 [B, Hkv, cap, D], then ``params`` float32 [B, Hkv, cap, 2]
    = (min, step) per row, a row's value being min + code * step."""

    def __init__(self, batch, n_kv_heads, cache_cap, head_dim, device, fill=0):
        n = gemma_kv_cache_bytes(batch, n_kv_heads, cache_cap, head_dim, GEMMA_F_KV_INT8)
        if n == 0:
            raise ValueError("bad int8 cache shape")
        self.shape = (batch, n_kv_heads, cache_cap, head_dim)
        self.buf = torch.full((n,), fill, dtype=torch.uint8, device=device)
        rows = batch * n_kv_heads * cache_cap
        off = gemma_kv_codes_bytes(batch, n_kv_heads, cache_cap, head_dim)
        self.codes = self.buf[:rows * head_dim].view(batch, n_kv_heads, cache_cap, head_dim)
        self.params = self.buf[off:off + rows * 8].view(torch.float32).view(batch, n_kv_heads, cache_cap, 2)
        self.device = self.buf.device

    def data_ptr(self):
        return self.buf.data_ptr()

    def numel(self):
        return self.buf.numel()


def _kv_kind(k_cache, v_cache) -> int:
    """GEMMA_F_KV_INT8 when the caches are Int8KVCache buffers, else 0; both
    caches (v_cache may be None under K = V) must be of one kind."""
    q8 = isinstance(k_cache, Int8KVCache)
    if v_cache is not None and isinstance(v_cache, Int8KVCache) != q8:
        raise TypeError("k_cache and v_cache must both be Int8KVCache buffers or both bf16 tensors")
    return GEMMA_F_KV_INT8 if q8 else 0


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _scratch(n, device, stream):
    """A workspace of n bytes for a call on `stream` (None: the current one).
    Allocated on that stream: the allocator hands the memory on in the order of
    the stream it was allocated on, so that neither what ran there before nor
    what the block serves next, once the call has returned, overlaps the call's
    kernels."""
    if stream is None:
        return torch.empty(max(n, 1), dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(max(n, 1), dtype=torch.uint8, device=device)


def _bf16(t, name):
    if t is None or isinstance(t, Int8KVCache):
        return
    if t.dtype != torch.bfloat16 or not t.is_contiguous() or not t.is_cuda:
        raise TypeError("%s must be a contiguous bf16 CUDA tensor" % name)


def gemma_last_error() -> str:
    s = _last()
    return s.decode() if s else ""


def gemma_attn_prefill_workspace_size(batch, s_new, n_q_heads, n_kv_heads, head_dim, window) -> int:
    return int(_prefill_ws(batch, s_new, n_q_heads, n_kv_heads, head_dim, window))


def gemma_attn_prefill_workspace_size_cached(batch, s_new, n_q_heads, n_kv_heads, head_dim, window, cache_cap,
                                             flags=0) -> int:
    return int(_prefill_ws_cached(batch, s_new, n_q_heads, n_kv_heads, head_dim, window, cache_cap, flags))


def gemma_attn_prefill(q, k_new, v_new, k_cache, v_cache, *, window, rope_frac, rope_theta, scale,
                       out, seq_lens_before=None, lse=None, workspace=None, flags=0, stream=None):
    """q [B,S,Hq,D]; k_new/v_new [B,S,Hkv,D] (None if shared); caches [B,Hkv,cap,D]."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"),
                 (v_cache, "v_cache"), (out, "out")):
        _bf16(t, n)
    B, S, Hq, D = q.shape
    _, Hkv, cap, _ = k_cache.shape
    flags |= _kv_kind(k_cache, v_cache)
    if workspace is None:
        n = (gemma_attn_prefill_workspace_size_cached(B, S, Hq, Hkv, D, window, cap, flags)
             if seq_lens_before is not None or flags & GEMMA_F_SHARED
             else gemma_attn_prefill_workspace_size(B, S, Hq, Hkv, D, window))
        workspace = _scratch(n, q.device, stream)
    return _check(_prefill(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), cap,
                           _ptr(seq_lens_before), B, S, window, Hq, Hkv, D, rope_frac, rope_theta,
                           scale, _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), flags,
                           _stream(stream)))


def gemma_attn_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, window, max_seq_len) -> int:
    return int(_decode_ws(batch, n_q_heads, n_kv_heads, head_dim, window, max_seq_len))


def gemma_attn_decode(q, k_new, v_new, k_cache, v_cache, *, seq_lens, max_seq_len, window,
                      rope_frac, rope_theta, scale, out, workspace=None, flags=0, stream=None):
    """q [B,Hq,D]; k_new/v_new [B,Hkv,D] (None if shared); caches [B,Hkv,cap,D];
    seq_lens int32 [B] on the device (length including the new token)."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"),
                 (v_cache, "v_cache"), (out, "out")):
        _bf16(t, n)
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise TypeError("seq_lens must be an int32 CUDA tensor")
    B, Hq, D = q.shape
    _, Hkv, cap, _ = k_cache.shape
    flags |= _kv_kind(k_cache, v_cache)
    if workspace is None:
        n = gemma_attn_decode_workspace_size(B, Hq, Hkv, D, window, max_seq_len)
        workspace = _scratch(n, q.device, stream)
    return _check(_decode(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), cap,
                          _ptr(seq_lens), max_seq_len, B, window, Hq, Hkv, D, rope_frac,
                          rope_theta, scale, _ptr(out), _ptr(workspace), workspace.numel(), flags,
                          _stream(stream)))


def gemma_attn_decode_multi_workspace_size(batch, tokens, n_q_heads, n_kv_heads, head_dim, window, max_seq_len,
                                           cache_cap, flags=0) -> int:
    return int(_multi_ws(batch, tokens, n_q_heads, n_kv_heads, head_dim, window, max_seq_len, cache_cap, flags))


def gemma_attn_decode_multi(q, k_new, v_new, k_cache, v_cache, *, seq_lens, max_seq_len, window,
                            rope_frac, rope_theta, scale, out, workspace=None, flags=0, stream=None):
    """q [B,T,Hq,D]; k_new/v_new [B,T,Hkv,D] (None if shared); caches [B,Hkv,cap,D];
    seq_lens int32 [B] on the device (length including the T new tokens)."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"),
                 (v_cache, "v_cache"), (out, "out")):
        _bf16(t, n)
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise TypeError("seq_lens must be an int32 CUDA tensor")
    B, T, Hq, D = q.shape
    _, Hkv, cap, _ = k_cache.shape
    flags |= _kv_kind(k_cache, v_cache)
    if workspace is None:
        n = gemma_attn_decode_multi_workspace_size(B, T, Hq, Hkv, D, window, max_seq_len, cap, flags)
        workspace = _scratch(n, q.device, stream)
    return _check(_multi(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), cap,
                         _ptr(seq_lens), max_seq_len, B, T, window, Hq, Hkv, D, rope_frac,
                         rope_theta, scale, _ptr(out), _ptr(workspace), workspace.numel(), flags,
                         _stream(stream)))


def _paged_args(k_pool, page_table):
    if page_table.dtype != torch.int32 or not page_table.is_cuda or page_table.dim() != 2:
        raise TypeError("page_table must be an int32 CUDA tensor [batch, pages_per_seq]")
    n_pages, Hkv, page_size, _ = k_pool.shape
    return n_pages, Hkv, page_size, page_table.shape[1]


def gemma_attn_prefill_paged(q, k_new, v_new, k_pool, v_pool, page_table, *, rope_frac, rope_theta, scale, out,
                             seq_lens_before=None, lse=None, workspace=None, flags=0, stream=None):
    """Global layer on a paged cache: pools [n_pages, Hkv, page_size, D]
    (bf16, or Int8KVCache(n_pages, Hkv, page_size, D) buffers), page_table
    int32 [B, pages_per_seq] on the device."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"), (v_pool, "v_pool"),
                 (out, "out")):
        _bf16(t, n)
    B, S, Hq, D = q.shape
    n_pages, Hkv, ps, pps = _paged_args(k_pool, page_table)
    flags |= _kv_kind(k_pool, v_pool)
    if workspace is None:
        n = (gemma_attn_prefill_workspace_size_cached(B, S, Hq, Hkv, D, 0, ps * pps, flags)
             if seq_lens_before is not None or flags & GEMMA_F_SHARED
             else gemma_attn_prefill_workspace_size(B, S, Hq, Hkv, D, 0))
        workspace = _scratch(n, q.device, stream)
    return _check(_prefill_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _ptr(page_table),
                                 ps, pps, n_pages, _ptr(seq_lens_before), B, S, Hq, Hkv, D, rope_frac, rope_theta,
                                 scale, _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), flags,
                                 _stream(stream)))


def gemma_attn_decode_paged(q, k_new, v_new, k_pool, v_pool, page_table, *, seq_lens, max_seq_len, rope_frac,
                            rope_theta, scale, out, workspace=None, flags=0, stream=None):
    """Global-layer decode on a paged cache (see gemma_attn_prefill_paged)."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"), (v_pool, "v_pool"),
                 (out, "out")):
        _bf16(t, n)
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise TypeError("seq_lens must be an int32 CUDA tensor")
    B, Hq, D = q.shape
    n_pages, Hkv, ps, pps = _paged_args(k_pool, page_table)
    flags |= _kv_kind(k_pool, v_pool)
    if workspace is None:
        n = gemma_attn_decode_workspace_size(B, Hq, Hkv, D, 0, max_seq_len)
        workspace = _scratch(n, q.device, stream)
    return _check(_decode_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _ptr(page_table),
                                ps, pps, n_pages, _ptr(seq_lens), max_seq_len, B, Hq, Hkv, D, rope_frac,
                                rope_theta, scale, _ptr(out), _ptr(workspace), workspace.numel(), flags,
                                _stream(stream)))


def gemma_attn_decode_multi_paged(q, k_new, v_new, k_pool, v_pool, page_table, *, seq_lens, max_seq_len, rope_frac,
                                  rope_theta, scale, out, workspace=None, flags=0, stream=None):
    """Multi-token decode of a global layer on a paged cache: q [B,T,Hq,D],
    k_new/v_new [B,T,Hkv,D]; pools and page table as gemma_attn_prefill_paged."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_pool, "k_pool"), (v_pool, "v_pool"),
                 (out, "out")):
        _bf16(t, n)
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise TypeError("seq_lens must be an int32 CUDA tensor")
    B, T, Hq, D = q.shape
    n_pages, Hkv, ps, pps = _paged_args(k_pool, page_table)
    flags |= _kv_kind(k_pool, v_pool)
    if workspace is None:
        n = gemma_attn_decode_multi_workspace_size(B, T, Hq, Hkv, D, 0, max_seq_len, ps * pps, flags)
        workspace = _scratch(n, q.device, stream)
    return _check(_multi_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _ptr(page_table),
                               ps, pps, n_pages, _ptr(seq_lens), max_seq_len, B, T, Hq, Hkv, D, rope_frac,
                               rope_theta, scale, _ptr(out), _ptr(workspace), workspace.numel(), flags,
                               _stream(stream)))


def gemma_kv_share_bind(dst: gemma_kv_desc, src: gemma_kv_desc) -> int:
    return _check(_bind(ctypes.byref(dst), ctypes.byref(src)))


def gemma_layer_schedule(n_layers: int, ratio: int, n_shared: int = 0):
    g = (_I * n_layers)()
    s = (_I * n_layers)()
    _check(_sched(n_layers, ratio, n_shared, g, s))
    return [bool(x) for x in g], [int(x) for x in s]


def gemma_attn_visible_ranges(batch, s_new, window, ranges, seq_lens_before=None, stream=None):
    if ranges.dtype != torch.int32 or not ranges.is_cuda or ranges.numel() < batch * s_new * 3:
        raise TypeError("ranges must be an int32 CUDA tensor of batch*s_new*3 elements")
    return _check(_ranges(_ptr(seq_lens_before), batch, s_new, window, _ptr(ranges), _stream(stream)))


def gemma_attn_sync_status(stream=None) -> int:
    """Returns the status code (does not raise)."""
    return int(_sync(_stream(stream)))


def gemma_attn_set_wait_limit(max_ns: int) -> int:
    return _check(_wait(max_ns))


def gemma_attn_debug_drop_next_copy(enable: bool) -> int:
    return _check(_drop(int(bool(enable))))


GEMMA_KERNEL_PREFILL_ROPE = 0
GEMMA_KERNEL_PREFILL_ATTN = 1
GEMMA_KERNEL_DECODE_APPEND = 2
GEMMA_KERNEL_DECODE_SPLIT = 3
GEMMA_KERNEL_DECODE_COMBINE = 4
KERNEL_NAMES = {0: "prefill_rope", 1: "prefill_attn", 2: "decode_append", 3: "decode_split",
                4: "decode_combine"}

_prof = _sig("gemma_attn_profile", _I, [_I])
_prof_read = _sig("gemma_attn_profile_read", _I, [_I, ctypes.POINTER(ctypes.c_double),
                                                  ctypes.POINTER(ctypes.c_longlong)])
_tinfo = _sig("gemma_attn_debug_timeout_info", _I, [ctypes.POINTER(ctypes.c_longlong)])
EXPORTED += ["gemma_attn_profile", "gemma_attn_profile_read", "gemma_attn_debug_timeout_info"]


def gemma_attn_debug_timeout_info():
    """-> list of 8 ints describing the first bounded wait that gave up (cleared on read)."""
    buf = (ctypes.c_longlong * 8)()
    _check(_tinfo(buf))
    return [int(x) for x in buf]


def gemma_attn_profile(enable: bool) -> int:
    return _check(_prof(int(bool(enable))))


def gemma_attn_profile_read(kernel: int):
    """-> (total device ms, launches) of one kernel kind since profiling began."""
    ms = ctypes.c_double()
    n = ctypes.c_longlong()
    _check(_prof_read(kernel, ctypes.byref(ms), ctypes.byref(n)))
    return float(ms.value), int(n.value)


_decode_noalloc = _sig("gemma_attn_decode_noalloc", _I, [_P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I,
                                                         _I, _F, _F, _F, _P, ctypes.c_uint, _P])
EXPORTED += ["gemma_attn_decode_noalloc", "gemma_attn_decode_multi_workspace_size", "gemma_attn_decode_multi",
             "gemma_attn_decode_multi_paged"]
NOALLOC_SCRATCH_BYTES = 32 << 20


def gemma_attn_decode_noalloc(q, k_new, v_new, k_cache, v_cache, *, seq_lens, max_seq_len, window,
                              rope_frac, rope_theta, scale, out, flags=0, stream=None):
    """gemma_attn_decode for callers that cannot allocate device memory: the
    split-K scratch is the library's fixed 32 MiB array (shared by all calls;
    overlapping calls race). Same arguments as gemma_attn_decode without the
    workspace."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"),
                 (v_cache, "v_cache"), (out, "out")):
        _bf16(t, n)
    if seq_lens.dtype != torch.int32 or not seq_lens.is_cuda:
        raise TypeError("seq_lens must be an int32 CUDA tensor")
    B, Hq, D = q.shape
    _, Hkv, cap, _ = k_cache.shape
    flags |= _kv_kind(k_cache, v_cache)
    return _check(_decode_noalloc(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), cap,
                                  _ptr(seq_lens), max_seq_len, B, window, Hq, Hkv, D, rope_frac,
                                  rope_theta, scale, _ptr(out), flags, _stream(stream)))


# ------------------------------------------------- window plus sinks, pages, axes
GEMMA_ROPE_INTERLEAVED = 1  # pairs go to the axes in turn
GEMMA_ROPE_AXIS_LADDERS = 2  # every axis has the whole range of frequencies
GEMMA_ROPE_INVERSE = 4  # the opposite rotation: gradient and inverse

_LL = ctypes.c_longlong


class gemma_page_book(ctypes.Structure):
    _fields_ = [("page_table", _P), ("ref_count", _P), ("n_seqs", _I), ("pages_per_seq", _I), ("n_pages", _I),
                ("page_size", _I)]


class gemma_page_pool(ctypes.Structure):
    _fields_ = [("pool", _P), ("n_kv_heads", _I), ("head_dim", _I), ("flags", ctypes.c_uint)]


_BOOK = ctypes.POINTER(gemma_page_book)
_POOLS = ctypes.POINTER(gemma_page_pool)
_prefill_sinks = _sig("gemma_attn_prefill_sinks", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _I, _I, _I,
                                                       _I, _F, _F, _F, _P, _P, _P, _SZ, ctypes.c_uint, _P])
_decode_sinks_ws = _sig("gemma_attn_decode_sinks_workspace_size", _SZ, [_I, _I, _I, _I, _I, _I, _I])
_decode_sinks = _sig("gemma_attn_decode_sinks", _I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _I, _I, _I, _I, _I,
                                                     _I, _F, _F, _F, _P, _P, _SZ, ctypes.c_uint, _P])
_pages_ws = _sig("gemma_kv_pages_workspace_size", _SZ, [_I, _I, _I])
_pages_fork = _sig("gemma_kv_pages_fork", _I, [_BOOK, _P, _P])
_pages_reserve = _sig("gemma_kv_pages_reserve", _I, [_BOOK, _POOLS, _I, _P, _P, _P, _P, _SZ, _P])
_pages_trim = _sig("gemma_kv_pages_trim", _I, [_BOOK, _P, _I, _I, _P])
_pages_compact = _sig("gemma_kv_pages_compact", _I, [_BOOK, _POOLS, _I, _P, _P, _P, _SZ, _P])
_pages_copy = _sig("gemma_kv_pages_copy", _I, [_POOLS, _I, _I, _I, _P, _P, _I, _P])
_rope_axes = _sig("gemma_rope_axes", _I, [_P, _LL, _P, _LL, _P, _I, ctypes.POINTER(_I), _I, _I, _I, _I, _F, _P, _LL,
                                          _P, _LL, ctypes.c_uint, _P])
EXPORTED += ["gemma_attn_prefill_sinks", "gemma_attn_decode_sinks_workspace_size", "gemma_attn_decode_sinks",
             "gemma_kv_pages_workspace_size", "gemma_kv_pages_fork", "gemma_kv_pages_reserve", "gemma_kv_pages_trim",
             "gemma_kv_pages_compact", "gemma_kv_pages_copy", "gemma_rope_axes"]


# These calls may be issued every few microseconds, so their checks use the
# cheap accessors: get_device() for tensors, the raw current stream and device
# (a CUDA tensor has been seen, so CUDA is initialised).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _on(index, stream, what, call, *args):
    """`call` with `args` and a stream of device `index` (by default its
    current one), that device current."""
    if index < 0:
        raise TypeError("%s: tensors must be on a CUDA device" % what)
    if stream is None:
        raw = _raw_stream(index)
    elif stream.device.index == index:
        raw = stream.cuda_stream
    else:
        raise ValueError("%s: stream of %s, tensors on cuda:%d" % (what, stream.device, index))
    if _current_device() == index:
        return _check(call(*args, raw))
    with torch.cuda.device(index):
        return _check(call(*args, raw))


def _int32(**numbers):
    """Refuses numbers that a C int would not hold (ctypes keeps their low 32
    bits without a word)."""
    for name, x in numbers.items():
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError("%s %d does not fit in 32 bits" % (name, x))


def _need(t, name, dtype, shape, index):
    """The data pointer of a contiguous tensor of this type, shape and device."""
    if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor on device %d" % (name, dtype, index))
    if t.shape != shape:
        raise ValueError("%s has shape %s, not %s" % (name, tuple(t.shape), tuple(shape)))
    return t.data_ptr()


_BF16, _I32 = torch.bfloat16, torch.int32


def _sinks_args(q, k_new, v_new, k_pool, v_pool, page_table, out, lens, lens_name, flags):
    """Shapes and devices of a window-plus-sinks call: its leading C arguments
    (q .. lens), (B, Hq, Hkv, D, capacity), out's pointer and the flags."""
    if isinstance(k_pool, Int8KVCache) or isinstance(v_pool, Int8KVCache):
        flags |= _kv_kind(k_pool, v_pool)  # refused below, by the library
        pools = (k_pool.data_ptr(), None if v_pool is None else v_pool.data_ptr())
    else:
        pools = None
    i = q.get_device()
    qs = q.shape
    B, Hq, D = qs[0], qs[-2], qs[-1]
    if len(k_pool.shape) != 4 or k_pool.shape[3] != D:
        raise ValueError("k_pool must be [n_pages, Hkv, page_size, D] with the D of q")
    n_pages, Hkv, ps, _ = shape = tuple(k_pool.shape)
    if pools is None:
        pools = (_need(k_pool, "k_pool", _BF16, shape, i),
                 None if v_pool is None else _need(v_pool, "v_pool", _BF16, shape, i))
    pps = page_table.shape[-1]
    new = (*qs[:-2], Hkv, D)
    args = (_need(q, "q", _BF16, qs, i), None if k_new is None else _need(k_new, "k_new", _BF16, new, i),
            None if v_new is None else _need(v_new, "v_new", _BF16, new, i), *pools,
            _need(page_table, "page_table", _I32, (B, pps), i), ps, pps, n_pages,
            None if lens is None else _need(lens, lens_name, _I32, (B,), i))
    return i, args, (B, Hq, Hkv, D), _need(out, "out", _BF16, qs, i), flags


def _workspace(workspace, size, index, stream):
    """(tensor, pointer, bytes) of the caller's workspace, or of one of size() bytes."""
    if workspace is None:
        n = size()
        if n == 0:
            return None, None, 0
        workspace = _scratch(n, "cuda:%d" % index, stream)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous tensor on device %d" % index)
    return workspace, workspace.data_ptr(), workspace.nbytes


def gemma_attn_prefill_sinks(q, k_new, v_new, k_pool, v_pool, page_table, *, window, sinks, rope_frac, rope_theta,
                             scale, out, seq_lens_before=None, lse=None, workspace=None, flags=0, stream=None):
    """A chunk on a paged layer that sees the last `window` positions and the
    first `sinks`: tensors as gemma_attn_prefill_paged (bf16 pools)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, S, Hq, D]")
    _int32(window=window, sinks=sinks)
    i, args, (B, Hq, Hkv, D), out_p, flags = _sinks_args(q, k_new, v_new, k_pool, v_pool, page_table, out,
                                                         seq_lens_before, "seq_lens_before", flags)
    S = q.shape[1]
    lse_p = None if lse is None else _need(lse, "lse", torch.float32, (B, Hq, S), i)
    keep, ws, ws_bytes = _workspace(workspace, lambda: gemma_attn_prefill_workspace_size(B, S, Hq, Hkv, D, 0), i, stream)
    return _on(i, stream, "gemma_attn_prefill_sinks", _prefill_sinks, *args, B, S, window, sinks, Hq, Hkv, D, rope_frac,
               rope_theta, scale, out_p, lse_p, ws, ws_bytes, flags)


def gemma_attn_decode_sinks_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, window, sinks, max_seq_len) -> int:
    return int(_decode_sinks_ws(batch, n_q_heads, n_kv_heads, head_dim, window, sinks, max_seq_len))


def gemma_attn_decode_sinks(q, k_new, v_new, k_pool, v_pool, page_table, *, seq_lens, max_seq_len, window, sinks,
                            rope_frac, rope_theta, scale, out, workspace=None, flags=0, stream=None):
    """One new token per sequence on a paged layer that sees the last `window`
    positions and the first `sinks`: tensors as gemma_attn_decode_paged (bf16
    pools); seq_lens 0 marks an idle slot."""
    if seq_lens is None:
        raise TypeError("seq_lens is required")
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    _int32(window=window, sinks=sinks, max_seq_len=max_seq_len)
    i, args, (B, Hq, Hkv, D), out_p, flags = _sinks_args(q, k_new, v_new, k_pool, v_pool, page_table, out, seq_lens,
                                                         "seq_lens", flags)
    keep, ws, ws_bytes = _workspace(
        workspace, lambda: gemma_attn_decode_sinks_workspace_size(B, Hq, Hkv, D, window, sinks, max_seq_len), i, stream)
    return _on(i, stream, "gemma_attn_decode_sinks", _decode_sinks, *args, max_seq_len, B, window, sinks, Hq, Hkv, D,
               rope_frac, rope_theta, scale, out_p, ws, ws_bytes, flags)


class PageBook:
    """Page table and reference counts of a paged cache, on the device:
    ``page_table`` int32 [n_seqs, pages_per_seq] (-1: no page) and
    ``ref_count`` int32 [n_pages], both views of ``state`` (one int32 tensor, so
    that a book is saved and restored with one copy). Starts empty."""

    def __init__(self, n_seqs, pages_per_seq, n_pages, page_size, device):
        n = n_seqs * pages_per_seq
        self.state = torch.zeros(n + n_pages, dtype=torch.int32, device=device)
        self.page_table = self.state[:n].view(n_seqs, pages_per_seq)
        self.ref_count = self.state[n:]
        self.page_table.fill_(-1)
        self.page_size = page_size
        self.n_seqs, self.pages_per_seq, self.n_pages = n_seqs, pages_per_seq, n_pages
        self.device = self.state.device
        self.desc = gemma_page_book(self.page_table.data_ptr(), self.ref_count.data_ptr(), n_seqs, pages_per_seq,
                                    n_pages, page_size)
        self._ref = ctypes.byref(self.desc)
        self._index = self.state.get_device()


def _pool_list(pools, n_pages, page_size, index):
    """gemma_page_pool array of bf16 tensors [n_pages, Hkv, page_size, D] and
    Int8KVCache(n_pages, Hkv, page_size, D) buffers."""
    rows = []
    for p in pools:
        q8 = isinstance(p, Int8KVCache)
        shape = p.shape
        if len(shape) != 4 or shape[0] != n_pages or shape[2] != page_size:
            raise ValueError("pool %d must be [n_pages %d, Hkv, page_size %d, D]" % (len(rows), n_pages, page_size))
        t = p.buf if q8 else p
        if t.get_device() != index or not (q8 or (t.dtype is _BF16 and t.is_contiguous())):
            raise TypeError("pool %d must be a contiguous bf16 tensor or an Int8KVCache on device %d" % (len(rows), index))
        rows.append((t.data_ptr(), shape[1], shape[3], GEMMA_F_KV_INT8 if q8 else 0))
    return (gemma_page_pool * max(len(rows), 1))(*rows)


def gemma_kv_pages_workspace_size(n_seqs, pages_per_seq, n_pages) -> int:
    return int(_pages_ws(n_seqs, pages_per_seq, n_pages))


def gemma_kv_pages_fork(book, parents, *, stream=None):
    """Row b of the book's table becomes row parents[b] (int32 [n_seqs]; b: unchanged, -1: empty)."""
    i = book._index
    return _on(i, stream, "gemma_kv_pages_fork", _pages_fork, book._ref,
               _need(parents, "parents", _I32, (book.n_seqs,), i))


def _book_workspace(book, workspace, stream):
    return _workspace(workspace, lambda: gemma_kv_pages_workspace_size(book.n_seqs, book.pages_per_seq, book.n_pages),
                      book._index, stream)


def gemma_kv_pages_reserve(book, pools, *, seq_lens, new_tokens, lacking, workspace=None, stream=None):
    """Grants pages (copying shared ones that will be written) for positions
    seq_lens[b] .. + new_tokens[b] of every row; lacking int32 [1] receives
    how many pages are missing (then nothing was changed)."""
    i, n = book._index, (book.n_seqs,)
    lens, new = _need(seq_lens, "seq_lens", _I32, n, i), _need(new_tokens, "new_tokens", _I32, n, i)
    short = _need(lacking, "lacking", _I32, (1,), i)
    arr = _pool_list(pools, book.n_pages, book.page_size, i)
    keep, ws, ws_bytes = _book_workspace(book, workspace, stream)
    return _on(i, stream, "gemma_kv_pages_reserve", _pages_reserve, book._ref, arr, len(pools), lens, new, short, ws,
               ws_bytes)


def gemma_kv_pages_trim(book, *, seq_lens, window=0, sinks=0, stream=None):
    """Drops the pages that hold nothing a token after seq_lens[b] sees
    (int32 [n_seqs]; 0 ends the sequence, below 0 leaves its row alone)."""
    _int32(window=window, sinks=sinks)
    i = book._index
    return _on(i, stream, "gemma_kv_pages_trim", _pages_trim, book._ref,
               _need(seq_lens, "seq_lens", _I32, (book.n_seqs,), i), window, sinks)


def gemma_kv_pages_compact(book, pools, *, n_live, page_map=None, workspace=None, stream=None):
    """Moves the live pages to numbers 0 .. n_live - 1 (n_live int32 [1],
    written); page_map int32 [n_pages]: the new number of every live page."""
    i = book._index
    live = _need(n_live, "n_live", _I32, (1,), i)
    names = None if page_map is None else _need(page_map, "page_map", _I32, (book.n_pages,), i)
    arr = _pool_list(pools, book.n_pages, book.page_size, i)
    keep, ws, ws_bytes = _book_workspace(book, workspace, stream)
    return _on(i, stream, "gemma_kv_pages_compact", _pages_compact, book._ref, arr, len(pools), live, names, ws, ws_bytes)


def gemma_kv_pages_copy(pools, *, src, dst, stream=None):
    """Copies pages src[i] -> dst[i] (int32 [n]) in every pool of the list."""
    if not pools:
        raise ValueError("no pools")
    n_pages, _, page_size, _ = pools[0].shape
    if src.dim() != 1:
        raise ValueError("src must be one-dimensional")
    i = src.get_device()
    src_p, dst_p = _need(src, "src", _I32, src.shape, i), _need(dst, "dst", _I32, src.shape, i)
    arr = _pool_list(pools, n_pages, page_size, i)
    return _on(i, stream, "gemma_kv_pages_copy", _pages_copy, arr, len(pools), n_pages, page_size, src_p, dst_p,
               src.shape[0])


def _token_stride(t, name, index):
    """Elements between tokens of a bf16 tensor [..., heads, D] on this device,
    whose heads are dense and whose tokens are evenly spaced."""
    if t.dtype is not _BF16 or t.get_device() != index:
        raise TypeError("%s must be a bf16 tensor on device %d" % (name, index))
    shape = t.shape
    D = shape[-1]
    if t.is_contiguous():
        return shape[-2] * D
    stride = t.stride()
    lead = [(n, s) for n, s in zip(shape[:-2], stride) if n != 1]
    if stride[-1] != 1 or (shape[-2] != 1 and stride[-2] != D) or any(
            s0 != n1 * s1 for (_, s0), (n1, s1) in zip(lead, lead[1:])):
        raise ValueError("%s: heads must be dense and tokens evenly spaced" % name)
    return lead[-1][1] if lead else shape[-2] * D


def gemma_rope_axes(q, k, positions, *, axis_pairs, rope_theta, q_out, k_out=None, flags=0, stream=None):
    """Rotary positions with several axes: q [..., Hq, D] and k [..., Hkv, D]
    (or None) turned by positions int32 [n_axes, ...] into q_out and k_out
    (which may be q and k). Tokens may be strided, e.g. slices of a fused
    projection; see GEMMA_ROPE_* for flags."""
    shape = q.shape
    if len(shape) < 3:
        raise ValueError("q must be [..., heads, head_dim]")
    i = q.get_device()
    *lead, Hq, D = shape
    if q_out.shape != shape:
        raise ValueError("q_out must have the shape of q")
    qs, qos = _token_stride(q, "q", i), _token_stride(q_out, "q_out", i)
    ks = kos = Hkv = 0
    k_p = ko_p = None
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    if k is not None:
        k_shape = k.shape
        *k_lead, Hkv, k_D = k_shape
        if k_lead != lead or k_D != D:
            raise ValueError("k has shape %s: tokens %s and head_dim %d expected" % (tuple(k_shape), tuple(lead), D))
        if k_out.shape != k_shape:
            raise ValueError("k_out must have the shape of k")
        ks, kos = _token_stride(k, "k", i), _token_stride(k_out, "k_out", i)
        k_p, ko_p = k.data_ptr(), k_out.data_ptr()
    n_axes, tokens = len(axis_pairs), math.prod(lead)
    _int32(tokens=tokens)
    pos = _need(positions, "positions", _I32, (n_axes, *lead), i)
    return _on(i, stream, "gemma_rope_axes", _rope_axes, q.data_ptr(), qs, k_p, ks, pos, n_axes,
               (_I * max(n_axes, 1))(*axis_pairs), tokens, Hq, Hkv, D, rope_theta, q_out.data_ptr(), qos, ko_p,
               kos, flags)
