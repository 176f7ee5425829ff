"""Python binding of the operators around a step's attention: the matrix product
with its epilogue (``include/dflash_linear.h``), the target's logits under
penalties, biases and masks (``include/dflash_logits.h``), and the pages of the
cache (``include/dflash_pages.h``).

The functions have the names of the C entry points and only marshal arguments.
``Linear`` owns a layer's handle; ``LogitsRules`` and ``PagePool`` hold the C
structures of what stays the same from call to call. Tensors that they hold are
read by later calls: what changes in the tensors of rules and pools is seen, a
layer's weights must stay as they are, and none may be freed or moved.
"""
from __future__ import annotations

import ctypes

from .paged import DFLASH_BF16, DFLASH_FP16, _binding, _empty_like_for, _int32, _one_device, _torch

DFLASH_FP32 = 3
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


class dflash_linear_config(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("w_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


class dflash_logits_rules(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("token_cols", ctypes.c_int32),
                ("lens", ctypes.c_void_p), ("prompt_lens", ctypes.c_void_p), ("repetition", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("temperature", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p), ("bias_stride", ctypes.c_int64),
                ("bias_count", ctypes.c_int32)]


class dflash_page_pool(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("counters", ctypes.c_void_p), ("requests", ctypes.c_int32),
                ("cols", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32)]


def declare(L):
    """Argument and result types of the entry points (those of a step are called through _step_call)."""
    P = ctypes.c_void_p
    L.dflash_linear_init.argtypes = [ctypes.POINTER(dflash_linear_config), P, P, P, ctypes.POINTER(P)]
    L.dflash_linear_sync_status.argtypes = [P, P]
    L.dflash_linear_destroy.argtypes = [P]
    I32 = ctypes.c_int32
    L.dflash_selftest_logits_lost.argtypes = [P, I32, I32, ctypes.c_int64, I32, ctypes.POINTER(dflash_logits_rules), P, P, P, I32, I32, P]
    for f in ("dflash_linear_init", "dflash_linear_sync_status", "dflash_linear_destroy", "dflash_selftest_logits_lost"):
        getattr(L, f).restype = ctypes.c_int


_calls = None


def _load_calls():
    """The helper module that marshals a step's calls (raises if it has not been built)."""
    global _calls
    L = _binding()[0]
    try:
        from . import _step_call
    except ImportError as e:
        raise RuntimeError("_step_call.so is missing: build it first (python -m "
                           "speculative_decoding_draft_tcgen05_gb300.build)") from e
    t = _torch()
    raw = getattr(t._C, "_cuda_getCurrentRawStream", None)  # device index -> handle of its current stream
    if raw is None:
        raw = lambda index: t.cuda.current_stream(index).cuda_stream  # noqa: E731
    at = [ctypes.cast(getattr(L, f), ctypes.c_void_p).value
          for f in ("dflash_linear_run", "dflash_logits_adjust", "dflash_pages_extend", "dflash_pages_trim",
                    "dflash_paged_current_device")]
    _step_call.setup(*at, raw, t.int32, t.float32, t.bfloat16, t.float16, t.int64)
    _calls = _step_call
    return _calls


# ------------------------------------------------------------ matrix product
class LinearHandle(ctypes.c_void_p):
    """The C handle with the shapes that it was made for."""


def dflash_linear_init(weight, bias=None, *, activation=None, out_dtype=None, stream=None):
    """Handle of y = residual + act(x weight^T + bias) for weight [n, k] and bias [n] (bfloat16 or float16, borrowed);
    activation None, "relu", "silu", "gelu" or "gelu_tanh"; out_dtype None (weight's) or torch.float32."""
    torch = _torch()
    L, check, get_stream = _binding()
    codes = {torch.bfloat16: DFLASH_BF16, torch.float16: DFLASH_FP16, torch.float32: DFLASH_FP32}
    out_dtype = weight.dtype if out_dtype is None else out_dtype
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {[a for a in ACTIVATIONS if a]}, got {activation!r}")
    if weight.dim() != 2 or (weight.shape[1] > 1 and weight.stride(1) != 1):
        raise ValueError("weight must be [n, k] with contiguous rows")
    if not weight.is_cuda or (bias is not None and not bias.is_cuda):
        raise ValueError("weight and bias must be CUDA tensors")
    n, k = weight.shape
    if bias is not None and (bias.dtype is not weight.dtype or tuple(bias.shape) != (n,) or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous {weight.dtype} [{n}], got {bias.dtype} {tuple(bias.shape)}")
    dev = _one_device(weight=weight, bias=bias)
    if dev != torch.cuda.current_device():
        raise ValueError(f"the weights are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    cfg = dflash_linear_config(n=n, k=k, w_stride=weight.stride(0), dtype=codes.get(weight.dtype, -1),
                               out_dtype=codes.get(out_dtype, -1), activation=ACTIVATIONS[activation])
    h = LinearHandle()
    check(L.dflash_linear_init(ctypes.byref(cfg), weight.data_ptr(), None if bias is None else bias.data_ptr(),
                               get_stream(stream), ctypes.cast(ctypes.byref(h), ctypes.POINTER(ctypes.c_void_p))),
          "dflash_linear_init")
    h.spec = (h.value, weight.dtype, out_dtype, n, k, dev)
    return h


def dflash_linear_run(handle, x, out, residual=None, stream=None):
    """out [rows, n] = residual + act(x weight^T + bias) for x [rows, k]; residual [rows, n] (out's dtype, may be out)."""
    st = (_calls or _load_calls()).linear(handle, x, out, residual, stream)
    if st:
        _binding()[1](st, "dflash_linear_run")


def dflash_linear_sync_status(handle, stream=None):
    """Waits for the stream; raises if a kernel latched an error."""
    L, check, get_stream = _binding()
    check(L.dflash_linear_sync_status(handle, get_stream(stream)), "dflash_linear_sync_status")


def dflash_linear_destroy(handle):
    """Frees the handle; calls with it are refused from then on."""
    L, check, _ = _binding()
    at = handle
    if isinstance(handle, LinearHandle):
        at, handle.value, handle.spec = handle.value, None, (0,) + handle.spec[1:]
    check(L.dflash_linear_destroy(at), "dflash_linear_destroy")


class Linear:
    """Owns a layer's handle and keeps its weights alive (convenience only). The weights must not change: a call may begin
    to read them before what was launched ahead of it has ended."""

    def __init__(self, weight, bias=None, *, activation=None, out_dtype=None, stream=None):
        self.h = None
        self.h = dflash_linear_init(weight, bias, activation=activation, out_dtype=out_dtype, stream=stream)
        self._weights = (weight, bias)  # the handle borrows them

    def __call__(self, x, out=None, *, residual=None, stream=None):
        if out is None:
            out = _empty_like_for(x, (x.shape[0], self.h.spec[3]), self.h.spec[2], stream)
        st = (_calls or _load_calls()).linear(self.h, x, out, residual, stream)
        if st:
            _binding()[1](st, "dflash_linear_run")
        return out

    def sync_status(self, stream=None):
        dflash_linear_sync_status(self.h, stream)

    def close(self):
        if self.h is not None:
            dflash_linear_destroy(self.h)  # (stays, empty: calls raise)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown
            pass


# ------------------------------------------------------------ logits
class LogitsRules:
    """What holds for each sequence of a batch (None: neutral): tokens [batch, cols] int32 so far, of which lens [batch]
    are valid and prompt_lens [batch] the prompt; repetition, presence, frequency and temperature [batch] fp32;
    bias_ids int32 and bias_values fp32 [batch, entries] (padding: an id outside the vocabulary)."""

    def __init__(self, tokens=None, lens=None, prompt_lens=None, *, repetition=None, presence=None, frequency=None,
                 temperature=None, bias_ids=None, bias_values=None):
        torch = _torch()
        vectors = dict(lens=lens, prompt_lens=prompt_lens, repetition=repetition, presence=presence, frequency=frequency,
                       temperature=temperature)
        matrices = dict(tokens=tokens, bias_ids=bias_ids, bias_values=bias_values)
        self.tensors = {n: t for n, t in {**vectors, **matrices}.items() if t is not None}
        if len({t.shape[0] for t in self.tensors.values()}) > 1:
            raise ValueError("tensors for different batches: " + ", ".join(f"{n} {tuple(t.shape)}" for n, t in self.tensors.items()))
        if tokens is not None and lens is None:
            raise ValueError("tokens need lens")
        if (bias_ids is None) != (bias_values is None) or (bias_ids is not None and bias_ids.shape != bias_values.shape):
            raise ValueError("bias_ids and bias_values must have the same shape")
        for n, t in self.tensors.items():
            dtype = torch.float32 if n in ("repetition", "presence", "frequency", "temperature", "bias_values") else torch.int32
            if t.dtype is not dtype:
                raise TypeError(f"{n} must be {dtype}, got {t.dtype}")
            if not t.is_cuda:
                raise ValueError(f"{n} must be a CUDA tensor")
            if t.dim() != (2 if n in matrices else 1) or (t.shape[-1] > 1 and t.stride(-1) != 1):
                raise ValueError(f"{n} must have {2 if n in matrices else 1} dimensions, the last one contiguous, got {tuple(t.shape)}")
        if bias_ids is not None and bias_ids.shape[0] > 1 and bias_ids.stride(0) != bias_values.stride(0):
            raise ValueError("bias_ids and bias_values must have the same strides")

        def at(t):
            return None if t is None else t.data_ptr()
        self.c = dflash_logits_rules(tokens=at(tokens), token_stride=0 if tokens is None else tokens.stride(0),
                                     token_cols=0 if tokens is None else tokens.shape[1], **{n: at(t) for n, t in vectors.items()},
                                     bias_ids=at(bias_ids), bias_values=at(bias_values),
                                     bias_stride=0 if bias_ids is None else bias_ids.stride(0),
                                     bias_count=0 if bias_ids is None else bias_ids.shape[1])
        self.spec = (ctypes.addressof(self.c), next((t.shape[0] for t in self.tensors.values()), -1), _one_device(**self.tensors))


def dflash_logits_adjust(logits, rules=None, *, out=None, probs=None, argmax=None, draft=None, mask=None, stream=None):
    """The rules on logits [batch, rows, vocab] (bfloat16, float16 or float32), whose position t follows draft [batch,
    rows - 1] int32 up to t; mask [batch, rows, ceil(vocab / 32)] int32 words (an expanded tensor shares them). Into any of
    out (like logits, may be them), probs [batch, rows, vocab] fp32 and argmax [batch, rows] int32."""
    st = (_calls or _load_calls()).logits(logits, rules, out, probs, argmax, draft, mask, stream)
    if st:
        _binding()[1](st, "dflash_logits_adjust")


def dflash_selftest_logits_lost(logits, rules=None, *, out=None, probs=None, argmax=None, rank, at, stream=None):
    """Self-test of the waits of dflash_logits_adjust: the logits of one CTA do not arrive from its position `at` on."""
    torch = _torch()
    if logits.dim() != 3:
        raise ValueError(f"logits must have 3 dimensions, got {tuple(logits.shape)}")
    for name, t, shape, dtype in (("logits", logits, logits.shape, logits.dtype), ("out", out, logits.shape, logits.dtype),
                                  ("probs", probs, logits.shape, torch.float32), ("argmax", argmax, logits.shape[:2], torch.int32)):
        if t is not None and (not t.is_cuda or not t.is_contiguous() or t.shape != shape or t.dtype is not dtype):
            raise ValueError(f"{name} must be a contiguous CUDA tensor {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    if rules is not None and rules.spec[1] not in (-1, logits.shape[0]):
        raise ValueError(f"the rules are for {rules.spec[1]} sequences, the logits for {logits.shape[0]}")
    dev = _one_device(logits=logits, out=out, probs=probs, argmax=argmax)
    if dev != torch.cuda.current_device() or (rules is not None and rules.spec[2] not in (-1, dev)):
        raise ValueError("the tensors must be on the current device")
    L, check, get_stream = _binding()
    code = {torch.bfloat16: DFLASH_BF16, torch.float16: DFLASH_FP16, torch.float32: DFLASH_FP32}.get(logits.dtype, -1)
    at_of = [None if t is None else t.data_ptr() for t in (out, probs, argmax)]
    check(L.dflash_selftest_logits_lost(logits.data_ptr(), *logits.shape, code, None if rules is None else ctypes.byref(rules.c),
                                        *at_of, rank, at, get_stream(stream)), "dflash_selftest_logits_lost")


# ------------------------------------------------------------ pages
class PagePool:
    """The pages behind a paged cache (int32 tensors): page_table [requests, cols], lens [requests] and the stack of
    free pages free_pages [num_pages], of which the first counters[0] are free (counters [2], the second 0)."""

    def __init__(self, page_table, lens, free_pages, counters, *, page_size):
        requests, cols = page_table.shape
        self.page_table, self.lens, self.free_pages, self.counters, self.page_size = page_table, lens, free_pages, counters, page_size
        self.c = dflash_page_pool(page_table=_int32(page_table, (requests, cols), "page_table"), table_stride=page_table.stride(0),
                                  lens=_int32(lens, (requests,), "lens"), free_pages=_int32(free_pages, (None,), "free_pages"),
                                  counters=_int32(counters, (2,), "counters"), requests=requests, cols=cols,
                                  page_size=page_size, num_pages=free_pages.shape[0])
        self.spec = (ctypes.addressof(self.c), requests,
                     _one_device(page_table=page_table, lens=lens, free_pages=free_pages, counters=counters))

    @classmethod
    def empty(cls, *, requests, cols, num_pages, page_size, device="cuda"):
        """A pool of which every page is free (page 0 is the first one taken)."""
        torch = _torch()
        kw = dict(device=device, dtype=torch.int32)
        return cls(torch.full((requests, cols), -1, **kw), torch.zeros(requests, **kw),
                   torch.arange(num_pages - 1, -1, -1, **kw), torch.tensor([num_pages, 0], **kw), page_size=page_size)

    def extend(self, batch, new_tokens, *, rows=None, positions=None, slots=None, granted=None, tokens=None, stream=None):
        """Gives the entries of `batch` (a PagedBatch whose tensors are written, or None) new_tokens [batch] more tokens,
        and writes their positions [tokens] int32 and slots [tokens] int64; rows [batch]: the entries' requests."""
        dflash_pages_extend(self, batch, new_tokens, rows=rows, positions=positions, slots=slots, granted=granted, tokens=tokens,
                            stream=stream)

    def trim(self, drop=None, *, accepted=None, drafts=None, rows=None, batch=None, stream=None):
        """Requests `rows` (None: the first ones) lose their last drop [batch] tokens; or, of blocks of `drafts` drafts,
        those that are not among the accepted [batch]; or, with neither, everything (`batch`: how many requests)."""
        if accepted is None:
            dflash_pages_trim(self, drop, rows=rows, batch=batch, stream=stream)
        elif drop is not None or drafts is None:
            raise ValueError("accepted goes with drafts, and not with drop")
        else:
            dflash_pages_trim(self, accepted, base=drafts, rows=rows, batch=batch, stream=stream)


def dflash_pages_extend(pool, batch, new_tokens, *, rows=None, positions=None, slots=None, granted=None, tokens=None, stream=None):
    """Pages, positions and slots of a batch's new tokens (PagePool.extend)."""
    st = (_calls or _load_calls()).extend(pool, batch, new_tokens, rows, positions, slots, granted, tokens, stream)
    if st:
        _binding()[1](st, "dflash_pages_extend")


def dflash_pages_trim(pool, counts=None, *, base=-1, rows=None, batch=None, stream=None):
    """Requests lose counts[b] tokens, base - counts[b] with base >= 0, everything with counts None (PagePool.trim)."""
    st = (_calls or _load_calls()).trim(pool, counts, rows, base, batch, stream)
    if st:
        _binding()[1](st, "dflash_pages_trim")
