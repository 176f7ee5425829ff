"""Python binding of the attention block's operators (``include/dflash_paged.h``):
per-head norm and rotation, append to a paged cache, attention over it.

The functions have the names of the C entry points and only marshal arguments.
``QkTransform``, ``PagedCache`` and ``PagedBatch`` hold the C structures of
what stays the same from call to call (a layer's weights, a layer's cache, a
step's batch); ``PagedAttention`` owns a handle. Tensors that they hold are
read by later calls: what changes in them (lengths, pages) is seen, but they
must not be freed or moved.
"""
from __future__ import annotations

import ctypes
import functools

DFLASH_BF16 = 0
DFLASH_FP16 = 1
DFLASH_E4M3 = 2


class dflash_paged_config(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32), ("cache_dtype", ctypes.c_int32),
                ("max_batch", ctypes.c_int32)]


class dflash_paged_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class dflash_paged_batch(ctypes.Structure):
    _fields_ = [("cu_tokens", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("table_cols", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("tokens", ctypes.c_int32), ("max_tokens", ctypes.c_int32)]


class dflash_qk_transform(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int64), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


def declare(L):
    """Argument and result types of the entry points (those of a step are called through _paged_call)."""
    P = ctypes.c_void_p
    L.dflash_paged_init.argtypes = [ctypes.POINTER(dflash_paged_config), P, ctypes.POINTER(P)]
    L.dflash_paged_sync_status.argtypes = [P, P]
    L.dflash_paged_destroy.argtypes = [P]
    for f in ("dflash_paged_init", "dflash_paged_sync_status", "dflash_paged_destroy"):
        getattr(L, f).restype = ctypes.c_int


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


@functools.lru_cache(maxsize=None)
def _binding():
    from . import _check, _stream, lib
    return lib(), _check, _stream


@functools.lru_cache(maxsize=None)
def _dtypes():
    t = _torch()
    return {t.bfloat16: DFLASH_BF16, t.float16: DFLASH_FP16, t.float8_e4m3fn: DFLASH_E4M3}


_calls = None


def _load_calls():
    """The helper module that marshals a step's calls (raises if it has not been built)."""
    global _calls
    L = _binding()[0]
    try:
        from . import _paged_call
    except ImportError as e:
        raise RuntimeError("_paged_call.so is missing: build it first (python -m "
                           "speculative_decoding_draft_tcgen05_gb300.build)") from e
    t = _torch()
    raw = getattr(t._C, "_cuda_getCurrentRawStream", None)  # device index -> handle of its current stream
    if raw is None:
        raw = lambda index: t.cuda.current_stream(index).cuda_stream  # noqa: E731
    at = [ctypes.cast(getattr(L, f), ctypes.c_void_p).value
          for f in ("dflash_qk_norm_rope", "dflash_paged_append", "dflash_paged_attend", "dflash_paged_current_device")]
    _paged_call.setup(*at, raw, t.int32, t.float32, t.bfloat16, t.float16)
    _calls = _paged_call
    return _calls


def _int32(t, shape, name):
    torch = _torch()
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return t.data_ptr()


def _one_device(**tensors):
    """The index of the device that all the given tensors (None: left out) are on; -1 without any."""
    at = {name: t.get_device() for name, t in tensors.items() if t is not None}
    if len(set(at.values())) > 1:
        raise ValueError("tensors on different devices: " + ", ".join(f"{n} on cuda:{i}" for n, i in at.items()))
    return next(iter(at.values()), -1)


class QkTransform:
    """Norm and rotation of query and key heads: table [positions, rotary_dim] fp32 (cosines, then sines; None: no
    rotation), norm weights [head_dim] of the calls' dtype (None: no norm)."""

    def __init__(self, table=None, *, rotary_dim=None, interleaved=False, q_weight=None, k_weight=None, eps=1e-6):
        torch = _torch()
        rotary_dim = (0 if table is None else table.shape[1]) if rotary_dim is None else rotary_dim
        if table is None and rotary_dim:
            raise ValueError("a rotation needs a table")
        if rotary_dim and (table.dim() != 2 or table.shape[1] != rotary_dim or not table.is_contiguous()
                           or not table.is_cuda):
            raise ValueError(f"table must be a contiguous CUDA tensor [positions, {rotary_dim}]")
        if rotary_dim and table.dtype is not torch.float32:
            raise TypeError(f"table must be torch.float32, got {table.dtype}")
        self.weights = [w for w in (q_weight, k_weight) if w is not None]
        for w in self.weights:
            if w.dim() != 1 or not w.is_contiguous() or not w.is_cuda:
                raise ValueError("norm weights must be contiguous CUDA tensors [head_dim]")
        if len({(w.dtype, w.shape) for w in self.weights}) > 1:
            raise TypeError("q_weight and k_weight must have the same dtype and size")
        self.table = table if rotary_dim else None  # kept alive with the addresses
        self.c = dflash_qk_transform(
            table=table.data_ptr() if rotary_dim else None, positions=table.shape[0] if rotary_dim else 0,
            rotary_dim=rotary_dim, interleaved=int(bool(interleaved)),
            q_weight=None if q_weight is None else q_weight.data_ptr(),
            k_weight=None if k_weight is None else k_weight.data_ptr(), eps=eps)
        w = self.weights[0] if self.weights else None
        self.spec = (ctypes.addressof(self.c), None if w is None else w.dtype, 0 if w is None else w.shape[0],
                     _one_device(table=self.table, q_weight=q_weight, k_weight=k_weight))


class PagedCache:
    """A layer's keys and values, each [num_pages, page_size, kv_heads, head_dim] (any strides with a contiguous last
    dimension, the same for both: a transposed [num_pages, kv_heads, page_size, head_dim] too). float8_e4m3fn
    caches hold value / scale."""

    def __init__(self, k, v, *, k_scale=1.0, v_scale=1.0):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype is not v.dtype:
            raise ValueError("k and v must be alike: [num_pages, page_size, kv_heads, head_dim], same strides and dtype")
        if k.dtype not in _dtypes():
            raise TypeError(f"a cache must be bfloat16, float16 or float8_e4m3fn, got {k.dtype}")
        if k.stride(3) != 1:
            raise ValueError("the cache's last dimension must be contiguous")
        if not (k.is_cuda and v.is_cuda):
            raise ValueError("k and v must be CUDA tensors")
        self.k, self.v = k, v
        page, slot, head = k.stride()[:3]
        self.c = dflash_paged_cache(k=k.data_ptr(), v=v.data_ptr(), num_pages=k.shape[0], page_stride=page,
                                    slot_stride=slot, head_stride=head if k.shape[2] > 1 else 0, k_scale=k_scale,
                                    v_scale=v_scale)
        self.spec = (ctypes.addressof(self.c), k.dtype, tuple(k.shape[1:]), _one_device(k=k, v=v))


class PagedBatch:
    """A step's batch: cu_tokens [batch + 1], lens [batch] (with the new tokens) and page_table [batch, cols], all
    int32 on the device; max_tokens: at least every sequence's number of new tokens."""

    def __init__(self, cu_tokens, lens, page_table, *, max_tokens):
        batch = lens.shape[0]
        self.tensors = (cu_tokens, lens, page_table)
        self.batch = batch
        self.c = dflash_paged_batch(cu_tokens=_int32(cu_tokens, (batch + 1,), "cu_tokens"),
                                    lens=_int32(lens, (batch,), "lens"),
                                    page_table=_int32(page_table, (batch, None), "page_table"),
                                    table_stride=page_table.stride(0), table_cols=page_table.shape[1], batch=batch,
                                    tokens=0, max_tokens=max_tokens)
        self.spec = (ctypes.addressof(self.c), _one_device(cu_tokens=cu_tokens, lens=lens, page_table=page_table))


def dflash_qk_norm_rope(q, k, q_out, k_out, transform, positions=None, stream=None):
    """q_out, k_out [tokens, heads, head_dim] = the transform of q and k (either pair may be None; in place is
    allowed); positions [tokens] int32."""
    st = (_calls or _load_calls()).norm_rope(q, k, q_out, k_out, transform, positions, stream)
    if st:
        _binding()[1](st, "dflash_qk_norm_rope")


class PagedHandle(ctypes.c_void_p):
    """The C handle with the shapes that it was made for."""


def dflash_paged_init(*, heads, kv_heads, head_dim, page_size, dtype, cache_dtype=None, max_batch, stream=None):
    """Handle of the attention operators for these shapes (torch dtypes; cache_dtype None: dtype)."""
    L, check, get_stream = _binding()
    codes = _dtypes()
    cfg = dflash_paged_config(heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size,
                              dtype=codes.get(dtype, -1),
                              cache_dtype=codes.get(dtype if cache_dtype is None else cache_dtype, -1),
                              max_batch=max_batch)
    h = PagedHandle()
    check(L.dflash_paged_init(ctypes.byref(cfg), get_stream(stream), ctypes.cast(ctypes.byref(h), ctypes.POINTER(ctypes.c_void_p))),
          "dflash_paged_init")
    h.spec = (h.value, dtype, dtype if cache_dtype is None else cache_dtype, heads, kv_heads, head_dim,
              (page_size, kv_heads, head_dim), _torch().cuda.current_device())
    return h


def dflash_paged_append(handle, cache, batch, k, v, transform=None, *, q=None, q_out=None, positions=None, stream=None):
    """Writes k (transformed) and v [tokens, kv_heads, head_dim] to the batch's places in the cache; with q also
    q_out = the transformed queries [tokens, heads, head_dim]."""
    st = (_calls or _load_calls()).append(handle, cache, batch, k, v, transform, q, q_out, positions, stream)
    if st:
        _binding()[1](st, "dflash_paged_append")


def dflash_paged_attend(handle, cache, batch, q, out, *, lse=None, causal=True, window=0, scale=None, stream=None):
    """out [tokens, heads, head_dim] = attention of q over the cache (scale None: 1 / sqrt(head_dim)); lse
    [tokens, heads] fp32."""
    st = (_calls or _load_calls()).attend(handle, cache, batch, q, out, lse, causal, window, scale, stream)
    if st:
        _binding()[1](st, "dflash_paged_attend")


def dflash_paged_sync_status(handle, stream=None):
    """Waits for the stream; raises if a kernel latched an error."""
    L, check, get_stream = _binding()
    check(L.dflash_paged_sync_status(handle, get_stream(stream)), "dflash_paged_sync_status")


def dflash_paged_destroy(handle):
    """Frees the handle; calls with it are refused from then on."""
    L, check, _ = _binding()
    at = handle
    if isinstance(handle, PagedHandle):
        at, handle.value, handle.spec = handle.value, None, (0,) + handle.spec[1:]
    check(L.dflash_paged_destroy(at), "dflash_paged_destroy")


def _empty_for(q, stream):
    """A tensor like q for a call on `stream`."""
    return _empty_like_for(q, q.shape, q.dtype, stream)


def _empty_like_for(q, shape, dtype, stream):
    """A tensor on q's device for a call on `stream` (None: the current one): memory that no earlier work of another
    stream may still touch, and that is not handed out again before the current stream's work up to then is done."""
    torch = _torch()
    if stream is not None:
        here = torch.cuda.current_stream(q.device)
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if handle != here.cuda_stream:
            with torch.cuda.stream(torch.cuda.ExternalStream(handle, q.device)):
                out = torch.empty(shape, dtype=dtype, device=q.device)
            out.record_stream(here)
            return out
    return torch.empty(shape, dtype=dtype, device=q.device)


class PagedAttention:
    """Owns a handle (convenience only)."""

    def __init__(self, *, heads, kv_heads, head_dim, page_size, dtype, cache_dtype=None, max_batch):
        self.h = None
        self.h = dflash_paged_init(heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, dtype=dtype,
                                   cache_dtype=cache_dtype, max_batch=max_batch)

    def append(self, cache, batch, k, v, transform=None, *, q=None, q_out=None, positions=None, stream=None):
        st = (_calls or _load_calls()).append(self.h, cache, batch, k, v, transform, q, q_out, positions, stream)
        if st:
            _binding()[1](st, "dflash_paged_append")

    def attend(self, cache, batch, q, out=None, *, lse=None, causal=True, window=0, scale=None, stream=None):
        if out is None:
            out = _empty_for(q, stream)
        st = (_calls or _load_calls()).attend(self.h, cache, batch, q, out, lse, causal, window, scale, stream)
        if st:
            _binding()[1](st, "dflash_paged_attend")
        return out

    def sync_status(self, stream=None):
        dflash_paged_sync_status(self.h, stream)

    def close(self):
        if self.h is not None:
            dflash_paged_destroy(self.h)  # (stays, empty: calls raise)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown
            pass
