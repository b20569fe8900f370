"""grouped_query_kv_gb300 -- Python binding of libkvattn (GB300 decode
attention over a grouped-query / multi-query KV cache).

The binding only marshals arguments: it checks dtypes, shapes, devices and
contiguity of torch tensors, and passes raw device pointers and the current
CUDA stream to the C ABI declared in ``include/kvattn.h``.  Every step of the
computation runs in the library's CUDA kernels; there is no CPU or PyTorch
fallback, and importing the entry points fails loudly if the compiled
library is missing (build it with ``python -m grouped_query_kv_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os
import threading


class _Torch:
    """torch, imported at the first use (which puts the module in this one's
    place): the library itself, its paths and its structures do without."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()

__all__ = [
    "kv_append", "kv_append_multi", "kv_append_paged", "gqa_decode_attn", "gqa_decode_step",
    "gqa_decode_attn_multi", "gqa_decode_attn_paged", "gqa_decode_step_paged",
    "kv_quantize_fp8", "kv_append_fp8", "gqa_decode_attn_fp8", "gqa_decode_step_fp8",
    "kv_block_tables", "kv_append_slots", "gqa_prefill_attn",
    "kv_append_paged_fp8", "gqa_decode_attn_paged_fp8",
    "check_device_error", "get_plan",
    "set_tuning", "set_wait_limit", "set_kernel_events", "release", "KvAttnError", "library_path", "lib",
    "KVATTN_OK", "KVATTN_ERR_INVALID_ARG", "KVATTN_ERR_UNSUPPORTED",
    "KVATTN_ERR_CUDA", "KVATTN_ERR_OOM", "KVATTN_ERR_DEVICE_BOUNDS",
    "KVATTN_ERR_TIMEOUT", "EXPORTED_SYMBOLS",
]

KVATTN_OK = 0
KVATTN_ERR_INVALID_ARG = 1
KVATTN_ERR_UNSUPPORTED = 2
KVATTN_ERR_CUDA = 3
KVATTN_ERR_OOM = 4
KVATTN_ERR_DEVICE_BOUNDS = 5
KVATTN_ERR_TIMEOUT = 6

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libkvattn.so")
_lock = threading.Lock()
_lib = None


class KvAttnError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__("%s (%d): %s" % (_status_name(status), status, detail))


class kvattn_plan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("tile_positions", ctypes.c_int),
                ("heads_per_cta", ctypes.c_int), ("head_groups", ctypes.c_int),
                ("stages", ctypes.c_int), ("threads", ctypes.c_int),
                ("num_ctas", ctypes.c_int), ("smem_bytes", ctypes.c_int),
                ("workspace_bytes", ctypes.c_int64)]


# name -> (restype, argtypes); mirrors include/kvattn.h
_VP = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong
_SIGS = {
    "kv_append": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP]),
    "kv_append_multi": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP]),
    "gqa_decode_attn": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                             ctypes.c_float, _VP]),
    "gqa_decode_step": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                             ctypes.c_float, _VP]),
    "gqa_decode_attn_multi": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                                   ctypes.c_float, _VP]),
    "gqa_decode_attn_window": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                                    ctypes.c_float, _I, _VP]),
    "gqa_decode_step_window": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                                    ctypes.c_float, _I, _VP]),
    "gqa_decode_attn_noalloc": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                                     ctypes.c_float, _VP]),
    "kv_append_paged": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _VP]),
    "kv_quantize_fp8": (_I, [_VP, _VP, _VP, ctypes.c_longlong, _I, _VP]),
    "kv_append_fp8": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _VP]),
    "gqa_decode_attn_fp8": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I,
                                 ctypes.c_float, _VP]),
    "gqa_decode_step_fp8": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I,
                                 _I, ctypes.c_float, _VP]),
    "gqa_decode_attn_paged": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I,
                                   _I, ctypes.c_float, _VP]),
    "gqa_decode_step_paged": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I,
                                   _I, _I, _I, ctypes.c_float, _VP]),
    "gqa_decode_attn_multi_window": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                                          ctypes.c_float, _I, _VP]),
    "gqa_decode_attn_paged_window": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                                          _I, _I, ctypes.c_float, _I, _VP]),
    "gqa_decode_step_paged_window": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I,
                                          _I, _I, _I, _I, ctypes.c_float, _I, _VP]),
    "kv_block_tables": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _VP]),
    "kv_append_slots": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _LL, _LL, _I, _I, _VP]),
    "gqa_prefill_attn": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _LL, _LL, _LL,
                              ctypes.c_float, _I, _VP]),
    "kv_append_paged_fp8": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I,
                                 _LL, _LL, _I, _I, _I, _VP]),
    "gqa_decode_attn_paged_fp8": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I,
                                       _I, _I, _I, ctypes.c_float, _VP]),
    "kvattn_status_string": (ctypes.c_char_p, [_I]),
    "kvattn_last_error": (ctypes.c_char_p, []),
    "kvattn_check_device_error": (_I, [_VP]),
    "kvattn_release": (None, []),
    "kvattn_set_tuning": (_I, [_I, _I]),
    "kvattn_set_wait_limit": (_I, [ctypes.c_uint]),
    "kvattn_set_kernel_events": (_I, [_VP, _VP]),
    "kvattn_get_plan": (_I, [_I, _I, _I, _I, _I, _I, ctypes.POINTER(kvattn_plan)]),
}
EXPORTED_SYMBOLS = tuple(_SIGS)


def library_path() -> str:
    return _LIB_PATH


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    h = _lib
    if h is not None:  # per-call fast path: no lock once loaded
        return h
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise ImportError(
                    "libkvattn.so is not built (%s); run "
                    "`python -m grouped_query_kv_gb300.build`" % _LIB_PATH)
            h = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in _SIGS.items():
                fn = getattr(h, name)
                fn.restype = res
                fn.argtypes = args
            _lib = h
    return _lib


def _status_name(status: int) -> str:
    try:
        return lib().kvattn_status_string(status).decode()
    except Exception:  # library not loadable: still give a readable error
        return "status"


def _check(status: int):
    if status != KVATTN_OK:
        raise KvAttnError(status, lib().kvattn_last_error().decode())


def _raw_stream(dev):
    # the current stream's handle without building a torch.cuda.Stream (several
    # microseconds of a decode step's host time), where torch has it
    global _raw_stream
    _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                   or (lambda d: torch.cuda.current_stream(d).cuda_stream))
    return _raw_stream(dev)


def _device():
    # the current device without torch.cuda's own call around it
    global _device
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _device()


def _stream_ptr(stream):
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream  # a plain int: ctypes converts it for the c_void_p argument


def _ptr(t):
    return t.data_ptr()


def _need(t, name, dtype, shape=None):
    # the checks run on every call of a decode loop, so they use the cheapest
    # torch attributes (is_cuda, dtype identity, torch.Size == tuple)
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (got %s)" % (name, t.device))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and t.shape != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))


def kv_append(k_cache, v_cache, k_new, v_new, seq_lens, stream=None):
    """Write the new token's K/V rows into row seq_lens[b] of the caches.

    k_cache, v_cache: bf16 [B, Hkv, Lmax, D] (in place); k_new, v_new: bf16
    [B, Hkv, D]; seq_lens: int32 [B], tokens cached before this one (not
    modified).
    """
    _need(k_cache, "k_cache", torch.bfloat16)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [B, Hkv, Lmax, D]")
    B, Hkv, Lmax, D = k_cache.shape
    _need(v_cache, "v_cache", torch.bfloat16, (B, Hkv, Lmax, D))
    _need(k_new, "k_new", torch.bfloat16, (B, Hkv, D))
    _need(v_new, "v_new", torch.bfloat16, (B, Hkv, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _check(lib().kv_append(_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                           _ptr(seq_lens), B, Hkv, D, Lmax, _stream_ptr(stream)))


def kv_append_multi(k_cache, v_cache, k_new, v_new, seq_lens, stream=None):
    """Write T new tokens' K/V rows: token t into row seq_lens[b] + t.

    k_cache, v_cache: bf16 [B, Hkv, Lmax, D] (in place); k_new, v_new: bf16
    [B, T, Hkv, D]; seq_lens: int32 [B], tokens cached before them (not
    modified).
    """
    _need(k_cache, "k_cache", torch.bfloat16)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [B, Hkv, Lmax, D]")
    B, Hkv, Lmax, D = k_cache.shape
    _need(v_cache, "v_cache", torch.bfloat16, (B, Hkv, Lmax, D))
    _need(k_new, "k_new", torch.bfloat16)
    if k_new.dim() != 4 or k_new.shape[0] != B or k_new.shape[2:] != (Hkv, D):
        raise ValueError("k_new must be [B, T, Hkv, D]")
    T = k_new.shape[1]
    _need(v_new, "v_new", torch.bfloat16, (B, T, Hkv, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _check(lib().kv_append_multi(_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new),
                                 _ptr(seq_lens), B, T, Hkv, D, Lmax, _stream_ptr(stream)))


def gqa_decode_attn(q, k_cache, v_cache, seq_lens, scale, out=None, stream=None,
                    window=None):
    """out[b,h] = softmax(scale * q[b,h] . K[b,h//G]^T) . V[b,h//G] over the
    first seq_lens[b] cached positions (only the last `window` of them for a
    local attention layer).

    q: bf16 [B, Hq, D]; caches: bf16 [B, Hkv, Lmax, D]; seq_lens: int32 [B];
    out: optional fp32 [B, Hq, D] (allocated if None); window: None (all
    positions) or an int >= 1.  Returns out.
    """
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    _need(k_cache, "k_cache", torch.bfloat16)
    if k_cache.dim() != 4 or k_cache.shape[0] != B or k_cache.shape[3] != D:
        raise ValueError("k_cache must be [B, Hkv, Lmax, D] matching q")
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    _need(v_cache, "v_cache", torch.bfloat16, (B, Hkv, Lmax, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, (B, Hq, D))
    if window is None:
        _check(lib().gqa_decode_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
                                     _ptr(out), B, Hq, Hkv, D, Lmax, float(scale),
                                     _stream_ptr(stream)))
    else:
        _check(lib().gqa_decode_attn_window(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                            _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D, Lmax,
                                            float(scale), _window(window), _stream_ptr(stream)))
    return out


def gqa_decode_step(q, k_new, v_new, k_cache, v_cache, seq_lens, scale, out=None,
                    stream=None, window=None):
    """One fused decode step: write k_new/v_new into row seq_lens[b] of the
    caches, then attend over positions [0, seq_lens[b] + 1) (only the last
    `window` of them for a local attention layer).

    q: bf16 [B, Hq, D]; k_new, v_new: bf16 [B, Hkv, D]; caches: bf16
    [B, Hkv, Lmax, D] (modified in place); seq_lens: int32 [B], tokens cached
    before this step (not modified); out: optional fp32 [B, Hq, D].
    """
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    _need(k_cache, "k_cache", torch.bfloat16)
    if k_cache.dim() != 4 or k_cache.shape[0] != B or k_cache.shape[3] != D:
        raise ValueError("k_cache must be [B, Hkv, Lmax, D] matching q")
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    _need(v_cache, "v_cache", torch.bfloat16, (B, Hkv, Lmax, D))
    _need(k_new, "k_new", torch.bfloat16, (B, Hkv, D))
    _need(v_new, "v_new", torch.bfloat16, (B, Hkv, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, (B, Hq, D))
    if window is None:
        _check(lib().gqa_decode_step(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D,
                                     Lmax, float(scale), _stream_ptr(stream)))
    else:
        _check(lib().gqa_decode_step_window(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                            _ptr(v_cache), _ptr(seq_lens), _ptr(out), B, Hq,
                                            Hkv, D, Lmax, float(scale), _window(window),
                                            _stream_ptr(stream)))
    return out


def gqa_decode_attn_multi(q, k_cache, v_cache, seq_lens, scale, out=None, stream=None,
                          window=None):
    """Attention for T new tokens per sequence, causal among themselves: token
    t of sequence b attends positions [0, e) with e = seq_lens[b] - T + 1 + t
    (only [e - window, e) for a local attention layer).

    q: bf16 [B, T, Hq, D]; caches: bf16 [B, Hkv, Lmax, D] already holding the
    new tokens' rows; seq_lens: int32 [B], tokens in the cache including the
    new ones; out: optional fp32 [B, T, Hq, D]; window: None (all positions)
    or an int >= 1.  Returns out.
    """
    _need(q, "q", torch.bfloat16)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D]")
    B, T, Hq, D = q.shape
    _need(k_cache, "k_cache", torch.bfloat16)
    if k_cache.dim() != 4 or k_cache.shape[0] != B or k_cache.shape[3] != D:
        raise ValueError("k_cache must be [B, Hkv, Lmax, D] matching q")
    Hkv, Lmax = k_cache.shape[1], k_cache.shape[2]
    _need(v_cache, "v_cache", torch.bfloat16, (B, Hkv, Lmax, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, T, Hq, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, (B, T, Hq, D))
    if window is None:
        _check(lib().gqa_decode_attn_multi(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                           _ptr(seq_lens), _ptr(out), B, T, Hq, Hkv, D, Lmax,
                                           float(scale), _stream_ptr(stream)))
    else:
        _check(lib().gqa_decode_attn_multi_window(_ptr(q), _ptr(k_cache), _ptr(v_cache),
                                                  _ptr(seq_lens), _ptr(out), B, T, Hq, Hkv, D,
                                                  Lmax, float(scale), _window(window),
                                                  _stream_ptr(stream)))
    return out


def _pool_shape(k_pool, block_table, name="k_pool"):
    """(num_blocks, Hkv, block_size, D, B, max_blocks) of a paged cache."""
    _need(k_pool, name, torch.bfloat16)
    if k_pool.dim() != 4:
        raise ValueError("%s must be [num_blocks, Hkv, block_size, D]" % name)
    _need(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    return tuple(k_pool.shape) + tuple(block_table.shape)


def kv_append_paged(k_pool, v_pool, k_new, v_new, block_table, seq_lens, stream=None):
    """Write new K/V rows into a paged pool: token t of sequence b goes to
    position seq_lens[b] + t, i.e. row (seq_lens[b] + t) % block_size of block
    block_table[b, (seq_lens[b] + t) // block_size].

    k_pool, v_pool: bf16 [num_blocks, Hkv, block_size, D] (in place);
    k_new, v_new: bf16 [B, Hkv, D] (one token) or [B, T, Hkv, D];
    block_table: int32 [B, max_blocks]; seq_lens: int32 [B], tokens cached
    before the new ones (not modified).
    """
    nblk, Hkv, bs, D, B, maxb = _pool_shape(k_pool, block_table)
    _need(v_pool, "v_pool", torch.bfloat16, (nblk, Hkv, bs, D))
    _need(k_new, "k_new", torch.bfloat16)
    if k_new.dim() == 3:
        T = 1
    elif k_new.dim() == 4:
        T = k_new.shape[1]
    else:
        raise ValueError("k_new must be [B, Hkv, D] or [B, T, Hkv, D]")
    if k_new.shape[0] != B or tuple(k_new.shape[-2:]) != (Hkv, D):
        raise ValueError("k_new must be [B, (T,) Hkv, D] matching the pool")
    _need(v_new, "v_new", torch.bfloat16, tuple(k_new.shape))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _check(lib().kv_append_paged(_ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new),
                                 _ptr(block_table), _ptr(seq_lens), B, T, Hkv, D, nblk, bs,
                                 maxb, _stream_ptr(stream)))


def gqa_decode_attn_paged(q, k_pool, v_pool, block_table, seq_lens, scale, out=None,
                          stream=None, window=None):
    """gqa_decode_attn (q [B, Hq, D]) or gqa_decode_attn_multi (q [B, T, Hq, D])
    over a paged cache: position j of sequence b is row j % block_size of
    block block_table[b, j // block_size] of the pools.

    k_pool, v_pool: bf16 [num_blocks, Hkv, block_size, D]; block_table: int32
    [B, max_blocks]; seq_lens: int32 [B]; out: optional fp32 shaped like q;
    window: None (all positions) or an int >= 1, each query's local window.
    Returns out.
    """
    _need(q, "q", torch.bfloat16)
    if q.dim() not in (3, 4):
        raise ValueError("q must be [B, Hq, D] or [B, T, Hq, D]")
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    T = 1 if q.dim() == 3 else q.shape[1]
    nblk, Hkv, bs, Dp, Bt, maxb = _pool_shape(k_pool, block_table)
    if Dp != D or Bt != B:
        raise ValueError("k_pool / block_table do not match q")
    _need(v_pool, "v_pool", torch.bfloat16, (nblk, Hkv, bs, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty(tuple(q.shape), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, tuple(q.shape))
    if window is None:
        _check(lib().gqa_decode_attn_paged(_ptr(q), _ptr(k_pool), _ptr(v_pool),
                                           _ptr(block_table), _ptr(seq_lens), _ptr(out), B, T,
                                           Hq, Hkv, D, nblk, bs, maxb, float(scale),
                                           _stream_ptr(stream)))
    else:
        _check(lib().gqa_decode_attn_paged_window(_ptr(q), _ptr(k_pool), _ptr(v_pool),
                                                  _ptr(block_table), _ptr(seq_lens), _ptr(out),
                                                  B, T, Hq, Hkv, D, nblk, bs, maxb,
                                                  float(scale), _window(window),
                                                  _stream_ptr(stream)))
    return out


def gqa_decode_step_paged(q, k_new, v_new, k_pool, v_pool, block_table, seq_lens, scale,
                          out=None, stream=None, window=None):
    """gqa_decode_step over a paged cache: the new token's rows go to position
    seq_lens[b] through the block table, then attention over [0, seq_lens[b] + 1)
    (only its last `window` positions for a local attention layer).

    q: bf16 [B, Hq, D]; k_new, v_new: bf16 [B, Hkv, D]; pools and table as
    for gqa_decode_attn_paged; seq_lens: tokens cached before this step.
    """
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    nblk, Hkv, bs, Dp, Bt, maxb = _pool_shape(k_pool, block_table)
    if Dp != D or Bt != B:
        raise ValueError("k_pool / block_table do not match q")
    _need(v_pool, "v_pool", torch.bfloat16, (nblk, Hkv, bs, D))
    _need(k_new, "k_new", torch.bfloat16, (B, Hkv, D))
    _need(v_new, "v_new", torch.bfloat16, (B, Hkv, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, (B, Hq, D))
    if window is None:
        _check(lib().gqa_decode_step_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_pool),
                                           _ptr(v_pool), _ptr(block_table), _ptr(seq_lens),
                                           _ptr(out), B, Hq, Hkv, D, nblk, bs, maxb,
                                           float(scale), _stream_ptr(stream)))
    else:
        _check(lib().gqa_decode_step_paged_window(_ptr(q), _ptr(k_new), _ptr(v_new),
                                                  _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                                  _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D,
                                                  nblk, bs, maxb, float(scale), _window(window),
                                                  _stream_ptr(stream)))
    return out


def kv_quantize_fp8(src, codes=None, scales=None, stream=None):
    """Quantize bf16 rows [..., D] into E4M3 codes (uint8 [..., D]) and one
    fp32 scale per row ([...]): scale = absmax / 448, code = E4M3(x / scale).
    Returns (codes, scales)."""
    _need(src, "src", torch.bfloat16)
    D = src.shape[-1]
    rows = src.numel() // D if D else 0
    if codes is None:
        codes = torch.empty(tuple(src.shape), dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty(tuple(src.shape[:-1]), dtype=torch.float32, device=src.device)
    _need(codes, "codes", torch.uint8, tuple(src.shape))
    _need(scales, "scales", torch.float32, tuple(src.shape[:-1]))
    _check(lib().kv_quantize_fp8(_ptr(src), _ptr(codes), _ptr(scales), rows, D,
                                 _stream_ptr(stream)))
    return codes, scales


def kv_append_fp8(k_codes, v_codes, k_scale, v_scale, k_new, v_new, seq_lens, stream=None):
    """Quantize the new token's K/V rows into position seq_lens[b] of an
    8-bit cache (codes uint8 [B, Hkv, Lmax, D], scales fp32 [B, Hkv, Lmax];
    k_new, v_new bf16 [B, Hkv, D])."""
    _need(k_codes, "k_codes", torch.uint8)
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [B, Hkv, Lmax, D]")
    B, Hkv, Lmax, D = k_codes.shape
    _need(v_codes, "v_codes", torch.uint8, (B, Hkv, Lmax, D))
    _need(k_scale, "k_scale", torch.float32, (B, Hkv, Lmax))
    _need(v_scale, "v_scale", torch.float32, (B, Hkv, Lmax))
    _need(k_new, "k_new", torch.bfloat16, (B, Hkv, D))
    _need(v_new, "v_new", torch.bfloat16, (B, Hkv, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    _check(lib().kv_append_fp8(_ptr(k_codes), _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
                               _ptr(k_new), _ptr(v_new), _ptr(seq_lens), B, Hkv, D, Lmax,
                               _stream_ptr(stream)))


def gqa_decode_attn_fp8(q, k_codes, v_codes, k_scale, v_scale, seq_lens, scale, out=None,
                        stream=None):
    """gqa_decode_attn over an 8-bit cache: K = E4M3(k_codes) * k_scale per
    row, V likewise.  q bf16 [B, Hq, D]; codes uint8 [B, Hkv, Lmax, D];
    scales fp32 [B, Hkv, Lmax]; seq_lens int32 [B]; out optional fp32
    [B, Hq, D].  Returns out."""
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    _need(k_codes, "k_codes", torch.uint8)
    if k_codes.dim() != 4 or k_codes.shape[0] != B or k_codes.shape[3] != D:
        raise ValueError("k_codes must be [B, Hkv, Lmax, D] matching q")
    Hkv, Lmax = k_codes.shape[1], k_codes.shape[2]
    _need(v_codes, "v_codes", torch.uint8, (B, Hkv, Lmax, D))
    _need(k_scale, "k_scale", torch.float32, (B, Hkv, Lmax))
    _need(v_scale, "v_scale", torch.float32, (B, Hkv, Lmax))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, (B, Hq, D))
    _check(lib().gqa_decode_attn_fp8(_ptr(q), _ptr(k_codes), _ptr(v_codes), _ptr(k_scale),
                                     _ptr(v_scale), _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D,
                                     Lmax, float(scale), _stream_ptr(stream)))
    return out


def gqa_decode_step_fp8(q, k_new, v_new, k_codes, v_codes, k_scale, v_scale, seq_lens, scale,
                        out=None, stream=None):
    """kv_append_fp8 then gqa_decode_attn_fp8 over seq_lens[b] + 1 positions,
    in one pass (the attention kernel writes the quantized rows first).
    q bf16 [B, Hq, D]; k_new, v_new bf16 [B, Hkv, D]; codes uint8
    [B, Hkv, Lmax, D] and scales fp32 [B, Hkv, Lmax], updated in place;
    seq_lens int32 [B] (tokens cached before this step, not modified);
    out optional fp32 [B, Hq, D].  Returns out."""
    _need(q, "q", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    _need(k_codes, "k_codes", torch.uint8)
    if k_codes.dim() != 4 or k_codes.shape[0] != B or k_codes.shape[3] != D:
        raise ValueError("k_codes must be [B, Hkv, Lmax, D] matching q")
    Hkv, Lmax = k_codes.shape[1], k_codes.shape[2]
    _need(v_codes, "v_codes", torch.uint8, (B, Hkv, Lmax, D))
    _need(k_scale, "k_scale", torch.float32, (B, Hkv, Lmax))
    _need(v_scale, "v_scale", torch.float32, (B, Hkv, Lmax))
    _need(k_new, "k_new", torch.bfloat16, (B, Hkv, D))
    _need(v_new, "v_new", torch.bfloat16, (B, Hkv, D))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.float32, (B, Hq, D))
    _check(lib().gqa_decode_step_fp8(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_codes),
                                     _ptr(v_codes), _ptr(k_scale), _ptr(v_scale),
                                     _ptr(seq_lens), _ptr(out), B, Hq, Hkv, D, Lmax,
                                     float(scale), _stream_ptr(stream)))
    return out


def _home(t, name):
    """The current CUDA device, which is where tensor t must be (the library
    launches there)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a CUDA tensor (got %s)" % (name, t.device))
    if dev != _device():
        raise ValueError("%s is on %s, not on the current CUDA device %d" % (name, t.device, _device()))
    return dev


def _on(stream, dev):
    """The handle of the stream to launch on, of device `dev` if None."""
    return _raw_stream(dev) if stream is None else _stream_ptr(stream)


def _want(t, name, dtype, dev, shape=None):
    """_need, and on CUDA device `dev`; one pass over the cheap attributes when
    all is well."""
    try:
        if (t.dtype is dtype and t.get_device() == dev and (shape is None or t.shape == shape)
                and t.is_contiguous()):
            return
    except AttributeError:
        pass
    _need(t, name, dtype, shape)
    raise ValueError("%s must be on the current CUDA device %d (got %s)" % (name, dev, t.device))


def _new(make, shape, dtype, like, stream):
    """An output made by torch.empty or torch.zeros on the stream that the call
    launches on, so that what fills it, or used its memory before, comes first."""
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    if not isinstance(stream, torch.cuda.Stream):  # (anything with the handle will do)
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


def _window(w):
    """w as a C int: what is beyond it attends everything, or is refused, as the
    nearest int that holds does (a window past every position, one below 1)."""
    return max(-0x80000000, min(int(w), 0x7fffffff))


def _int32(x, name):
    """x as an int that a C int holds."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError("%s is beyond 32 bits (%d)" % (name, x))
    return x


def _packed_rows(t, name, dev, shape=None):
    """Checks packed bf16 rows [N, H, D] whose [H, D] are contiguous (they may
    be a slice of wider rows) and returns the elements from row to row."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.get_device() != dev:
        raise ValueError("%s must be a CUDA tensor on the current device %d (got %s)" % (name, dev, t.device))
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s must be %s (got %s)" % (name, torch.bfloat16, t.dtype))
    if shape is None:
        if t.dim() != 3:
            raise ValueError("%s must be [N, heads, D]" % name)
        shape = t.shape
    elif t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, shape, tuple(t.shape)))
    N, H, D = shape
    row, head, one = t.stride()
    if (one != 1 and D > 1) or (head != D and H > 1):
        raise ValueError("%s: each row's [heads, D] must be contiguous (strides %s)" % (name, t.stride()))
    return row if N > 1 else H * D


def kv_block_tables(cached_lens, new_lens, block_table, free_blocks, free_count, block_size,
                    num_slots, cu_seqlens=None, slots=None, free_count_out=None, stream=None):
    """Blocks and slots for each request's new tokens, packed request after
    request: request b keeps its ceil(cached_lens[b] / block_size) blocks and
    takes the ones it lacks for new_lens[b] more tokens from the top of the
    free stack (free_blocks[:free_count]); packed row cu_seqlens[b] + i gets
    slot block * block_size + offset of position cached_lens[b] + i, rows
    behind the last token -1.

    cached_lens, new_lens: int32 [B]; block_table: int32 [B, max_blocks] (in
    place); free_blocks: int32 [num_free]; free_count: int32 [1]; num_slots:
    rows of the slot map.  cu_seqlens (int32 [B + 1]) and slots (int64
    [num_slots]) are allocated if None; the count left goes to free_count_out
    (None: back into free_count).  Returns (cu_seqlens, slots, free_count_out).
    Requests that the free list or the table cannot serve get slot -1 and set
    the device error word (see include/kvattn.h).
    """
    i32, dev = torch.int32, _home(cached_lens, "cached_lens")
    _want(cached_lens, "cached_lens", i32, dev)
    if cached_lens.dim() != 1:
        raise ValueError("cached_lens must be [B]")
    B = cached_lens.shape[0]
    _want(new_lens, "new_lens", i32, dev, (B,))
    _want(block_table, "block_table", i32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    _want(free_blocks, "free_blocks", i32, dev)
    if free_blocks.dim() != 1:
        raise ValueError("free_blocks must be [num_free]")
    _want(free_count, "free_count", i32, dev, (1,))
    num_slots = _int32(num_slots, "num_slots")
    if cu_seqlens is None:
        cu_seqlens = _new(torch.empty, (B + 1,), i32, cached_lens, stream)
    else:
        _want(cu_seqlens, "cu_seqlens", i32, dev, (B + 1,))
    if slots is None:
        slots = _new(torch.empty, (max(num_slots, 0),), torch.int64, cached_lens, stream)
    else:
        _want(slots, "slots", torch.int64, dev, (num_slots,))
    if free_count_out is None:
        free_count_out = free_count
    else:
        _want(free_count_out, "free_count_out", i32, dev, (1,))
    _check(lib().kv_block_tables(cached_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
                                 free_blocks.data_ptr(), free_count.data_ptr(), free_count_out.data_ptr(),
                                 cu_seqlens.data_ptr(), slots.data_ptr(), B, block_table.shape[1],
                                 _int32(block_size, "block_size"), free_blocks.shape[0], num_slots,
                                 _on(stream, dev)))
    return cu_seqlens, slots, free_count_out


def kv_append_slots(k_pool, v_pool, k_new, v_new, slots, stream=None):
    """Write packed K/V rows into a paged pool: row i goes to row
    slots[i] % block_size of block slots[i] // block_size; a negative slot
    skips its row.  At least one row.

    k_pool, v_pool: bf16 [num_blocks, Hkv, block_size, D] (in place); k_new,
    v_new: bf16 [N, Hkv, D], rows contiguous or slices of wider rows; slots:
    int64 [N], all different.
    """
    dev = _home(k_pool, "k_pool")
    _want(k_pool, "k_pool", torch.bfloat16, dev)
    if k_pool.dim() != 4:
        raise ValueError("k_pool must be [num_blocks, Hkv, block_size, D]")
    nblk, Hkv, bs, D = k_pool.shape
    _want(v_pool, "v_pool", torch.bfloat16, dev, (nblk, Hkv, bs, D))
    _want(slots, "slots", torch.int64, dev)
    if slots.dim() != 1:
        raise ValueError("slots must be [N]")
    N = slots.shape[0]
    ks = _packed_rows(k_new, "k_new", dev, (N, Hkv, D))
    vs = _packed_rows(v_new, "v_new", dev, (N, Hkv, D))
    _check(lib().kv_append_slots(k_pool.data_ptr(), v_pool.data_ptr(), k_new.data_ptr(),
                                 v_new.data_ptr(), slots.data_ptr(), N, Hkv, D, ks, vs, nblk, bs, _on(stream, dev)))


def gqa_prefill_attn(q, k, v, cu_seqlens, scale, out=None, stream=None, window=None):
    """Causal attention of whole prompts packed one after the other: token i
    of sequence b (rows [cu_seqlens[b], cu_seqlens[b + 1])) attends the rows
    j <= i of its sequence (j > i - window on a local attention layer).  Only
    these rows: it is for prompts with nothing cached, not for tokens that
    continue a cached prefix.

    q: bf16 [N, Hq, D]; k, v: bf16 [N, Hkv, D], rows contiguous or slices of
    wider rows; cu_seqlens: int32 [B + 1]; out: optional bf16 [N, Hq, D] (if
    None allocated as zeros, since rows of no sequence are not written);
    window: None (all positions) or an int >= 1.  Returns out.
    """
    dev = _home(q, "q")
    qs = _packed_rows(q, "q", dev)
    N, Hq, D = q.shape
    ks = _packed_rows(k, "k", dev)
    Hkv = k.shape[1]
    if k.shape[0] != N or k.shape[2] != D:
        raise ValueError("k must be [N, Hkv, D] matching q")
    vs = _packed_rows(v, "v", dev, (N, Hkv, D))
    _want(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if cu_seqlens.dim() != 1:
        raise ValueError("cu_seqlens must be [B + 1]")
    if out is None:
        out = _new(torch.zeros, (N, Hq, D), torch.bfloat16, q, stream)
    else:
        _want(out, "out", torch.bfloat16, dev, (N, Hq, D))
    _check(lib().gqa_prefill_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), out.data_ptr(),
                                  cu_seqlens.shape[0] - 1, N, Hq, Hkv, D, qs, ks, vs, float(scale),
                                  0x7fffffff if window is None else _window(window),
                                  _on(stream, dev)))
    return out


def _pool8(k_codes, v_codes, k_scale, v_scale, block_table, dev):
    """Checks a paged 8-bit cache; returns (num_blocks, Hkv, block_size, D, B, max_blocks)."""
    _want(k_codes, "k_codes", torch.uint8, dev)
    if k_codes.dim() != 4:
        raise ValueError("k_codes must be [num_blocks, Hkv, block_size, D]")
    nblk, Hkv, bs, D = k_codes.shape
    _want(v_codes, "v_codes", torch.uint8, dev, (nblk, Hkv, bs, D))
    _want(k_scale, "k_scale", torch.float32, dev, (nblk, Hkv))
    _want(v_scale, "v_scale", torch.float32, dev, (nblk, Hkv))
    _want(block_table, "block_table", torch.int32, dev)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    return nblk, Hkv, bs, D, block_table.shape[0], block_table.shape[1]


def kv_append_paged_fp8(k_codes, v_codes, k_scale, v_scale, k_new, v_new, block_table, cached_lens,
                        cu_seqlens, stream=None):
    """Quantize packed K/V rows into a paged 8-bit cache with one power-of-two
    scale per block and K/V head: token i of request b (packed row
    cu_seqlens[b] + i) goes to position cached_lens[b] + i of its table row.  A
    block's scale grows with its rows; earlier codes are rewritten for it.
    gqa_decode_attn_paged_fp8 reads such pools where D is 128 or 256.

    k_codes, v_codes: uint8 [num_blocks, Hkv, block_size, D]; k_scale,
    v_scale: fp32 [num_blocks, Hkv] (all in place); k_new, v_new: bf16
    [N, Hkv, D], rows contiguous or slices of wider rows; block_table: int32
    [B, max_blocks]; cached_lens: int32 [B]; cu_seqlens: int32 [B + 1].
    """
    dev = _home(k_codes, "k_codes")
    nblk, Hkv, bs, D, B, maxb = _pool8(k_codes, v_codes, k_scale, v_scale, block_table, dev)
    ks = _packed_rows(k_new, "k_new", dev)
    N = k_new.shape[0]
    if k_new.shape[1] != Hkv or k_new.shape[2] != D:
        raise ValueError("k_new must be [N, Hkv, D] matching the pool")
    vs = _packed_rows(v_new, "v_new", dev, (N, Hkv, D))
    _want(cached_lens, "cached_lens", torch.int32, dev, (B,))
    _want(cu_seqlens, "cu_seqlens", torch.int32, dev, (B + 1,))
    _check(lib().kv_append_paged_fp8(k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                     k_new.data_ptr(), v_new.data_ptr(), block_table.data_ptr(), cached_lens.data_ptr(),
                                     cu_seqlens.data_ptr(), B, N, Hkv, D, ks, vs, nblk, bs, maxb,
                                     _on(stream, dev)))


def gqa_decode_attn_paged_fp8(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, scale,
                              out=None, stream=None):
    """gqa_decode_attn over a paged 8-bit cache: K = E4M3(k_codes) *
    k_scale[block, kvh], V likewise.  q: bf16 [B, Hq, D]; pools and table as for
    kv_append_paged_fp8; seq_lens: int32 [B], positions attended; out: optional
    bf16 [B, Hq, D].  Returns out."""
    dev = _home(q, "q")
    _want(q, "q", torch.bfloat16, dev)
    if q.dim() != 3:
        raise ValueError("q must be [B, Hq, D]")
    B, Hq, D = q.shape
    nblk, Hkv, bs, Dp, Bt, maxb = _pool8(k_codes, v_codes, k_scale, v_scale, block_table, dev)
    if Dp != D or Bt != B:
        raise ValueError("k_codes / block_table do not match q")
    _want(seq_lens, "seq_lens", torch.int32, dev, (B,))
    if out is None:
        out = _new(torch.empty, (B, Hq, D), torch.bfloat16, q, stream)
    else:
        _want(out, "out", torch.bfloat16, dev, (B, Hq, D))
    _check(lib().gqa_decode_attn_paged_fp8(q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(), k_scale.data_ptr(),
                                           v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                                           out.data_ptr(), B, Hq, Hkv, D, nblk, bs, maxb, float(scale),
                                           _on(stream, dev)))
    return out


def check_device_error(stream=None):
    """Synchronise the stream and raise KvAttnError if the device flagged one."""
    _check(lib().kvattn_check_device_error(_stream_ptr(stream)))


def get_plan(B, Hq, Hkv, D, Lmax, num_sms=0) -> dict:
    p = kvattn_plan()
    _check(lib().kvattn_get_plan(B, Hq, Hkv, D, Lmax, num_sms, ctypes.byref(p)))
    return {name: getattr(p, name) for name, _ in kvattn_plan._fields_}


def set_tuning(force_path: int = 0, num_ctas: int = 0):
    _check(lib().kvattn_set_tuning(force_path, num_ctas))


def set_wait_limit(polls: int = 0):
    """Test knob: polls before the tensor-core kernel's pipeline waits give
    up (0 restores the default); see kvattn_set_wait_limit."""
    _check(lib().kvattn_set_wait_limit(int(polls)))


def set_kernel_events(before=None, after=None):
    """Measurement hook: record these torch.cuda.Event objects just before
    and just after the split-KV kernel of every later attention call (None,
    None stops).  The events must have been created (recorded once) first."""
    if (before is None) != (after is None):
        raise ValueError("give both events or neither")
    b = before.cuda_event if before is not None else None
    a = after.cuda_event if after is not None else None
    if before is not None and (not b or not a):
        raise ValueError("record each event once before handing it over (torch creates it lazily)")
    _check(lib().kvattn_set_kernel_events(b, a))


def release():
    lib().kvattn_release()
