"""The marshalling of the calls around a step's attention (csrc/step_call.c) and
the refusals of their entry points, on the CPU: a copy of the helper module
with recording entry points and stand-ins for tensors, which it knows only by
their attributes; and the library's own checks, which come before any launch."""
import ctypes
import importlib.util
import shutil

import pytest

P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
BF16, FP16, INT32, FLOAT32, INT64 = "bf16", "fp16", "int32", "float32", "int64"


class Tensor:
    def __init__(self, *shape, dtype=BF16, device=0, at=4096, strides=None):
        self.dtype, self.shape, self.device, self.at, self.strides = dtype, tuple(shape), device, at, strides

    def stride(self):
        if self.strides:
            return self.strides
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s)

    def get_device(self):
        return self.device

    def data_ptr(self):
        return self.at

    def is_contiguous(self):
        return self.strides is None


class Spec:
    def __init__(self, *spec):
        self.spec = spec


class Batch(ctypes.Structure):
    _fields_ = [("cu_tokens", P), ("lens", P), ("page_table", P), ("table_stride", I64), ("table_cols", I32), ("batch", I32),
                ("tokens", I32), ("max_tokens", I32)]


class Calls:
    """The module, with what its entry points were called with."""

    def __init__(self, path):
        spec = importlib.util.spec_from_file_location("_step_call", path)
        self.m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(self.m)
        self.made, self.now, self.keep = [], 0, []
        at = []
        for name, args in (("linear", [P, P, I64, I64, P, I64, P, I64, P]),
                           ("logits", [P, I64, I64, I32, I32, I64, I32, P, P, I64, P, I64, I64, P, I64, I64, P, P, P]),
                           ("extend", [P, P, P, I32, I32, P, P, P, I64, I32, P, P, P, P]), ("trim", [P, P, P, I32, I32, P])):
            f = ctypes.CFUNCTYPE(ctypes.c_int, *args)(lambda *a, name=name: self.made.append((name, a)) or 0)
            self.keep.append(f)
            at.append(ctypes.cast(f, P).value)
        f = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: self.now)
        self.keep.append(f)
        self.m.setup(*at, ctypes.cast(f, P).value, lambda index: 1000 + index, INT32, FLOAT32, BF16, FP16, INT64)
        self.c = ctypes.create_string_buffer(512)
        self.c_at = ctypes.addressof(self.c)
        self.b = Batch(cu_tokens=16, lens=32, page_table=48, table_stride=10, table_cols=10, batch=3)

    def handle(self, device=0):
        return Spec(self.c_at, BF16, FLOAT32, 32, 64, device)

    def pool(self, device=0):
        return Spec(self.c_at, 5, device)

    def batch(self, device=0):
        return Spec(ctypes.addressof(self.b), device)


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    from speculative_decoding_draft_tcgen05_gb300 import build
    build.build()
    at = tmp_path_factory.mktemp("call") / "_step_call.so"  # its own copy: the module's state is per file
    shutil.copy(build.STEP_CALL, at)
    return Calls(str(at))


@pytest.fixture(autouse=True)
def fresh(calls):
    calls.made.clear()
    calls.now = 0


def ints(*shape, device=0, **k):
    return Tensor(*shape, dtype=INT32, device=device, **k)


def test_linear(calls):
    x, y = Tensor(4, 64, at=64, strides=(80, 1)), Tensor(4, 32, dtype=FLOAT32, at=128)
    assert calls.m.linear(calls.handle(), x, y, None, None) == 0
    name, a = calls.made[0]
    assert a[1:4] == (64, 80, 4) and a[4] is None and a[6:8] == (128, 32) and a[8] == 1000
    assert calls.m.linear(calls.handle(), Tensor(1, 64, strides=(7, 1)), Tensor(1, 32, dtype=FLOAT32), Tensor(1, 32, dtype=FLOAT32), 77) == 0
    assert calls.made[1][1][2] == 64 and calls.made[1][1][8] == 77  # one row may carry any stride


@pytest.mark.parametrize("which", range(4))
def test_linear_refuses_tensors_of_two_devices(calls, which):
    at = [0] * 4
    at[which] = 1
    args = (calls.handle(at[0]), Tensor(4, 64, device=at[1]), Tensor(4, 32, dtype=FLOAT32, device=at[2]), Tensor(4, 32, dtype=FLOAT32, device=at[3]))
    with pytest.raises(ValueError, match="cuda:"):
        calls.m.linear(*args, None)
    assert not calls.made


def test_linear_refuses_other_shapes_and_types(calls):
    good = [calls.handle(), Tensor(4, 64), Tensor(4, 32, dtype=FLOAT32), None, None]
    for i, bad in ((1, Tensor(4, 63)), (1, Tensor(4, 64, dtype=FP16)), (1, Tensor(64)), (1, Tensor(4, 64, strides=(1, 4))),
                   (1, Tensor(4, 64, device=-1)), (2, Tensor(4, 32)), (2, Tensor(3, 32, dtype=FLOAT32)), (3, Tensor(4, 31, dtype=FLOAT32)),
                   (0, Spec(1, 2))):
        args = list(good)
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            calls.m.linear(*args)
    assert not calls.made


def test_logits(calls):
    x, out, probs, best = Tensor(2, 3, 65), Tensor(2, 3, 65), Tensor(2, 3, 65, dtype=FLOAT32), ints(2, 3)
    draft, mask = ints(2, 2), ints(2, 3, 3, strides=(0, 0, 1))
    rules = Spec(calls.c_at, 2, 0)
    assert calls.m.logits(x, rules, out, probs, best, draft, mask, None) == 0
    a = calls.made[0][1]
    assert a[1:7] == (195, 65, 2, 3, 65, 0) and a[9] == 2 and a[11:13] == (0, 0) and a[14:16] == (195, 65)
    assert calls.m.logits(Tensor(2, 1, 64, dtype=FLOAT32), None, None, None, ints(2, 1), None, None, None) == 0
    assert calls.made[1][1][6] == 3


@pytest.mark.parametrize("which", range(7))
def test_logits_refuses_tensors_of_two_devices(calls, which):
    at = [0] * 7
    at[which] = 1
    args = (Tensor(2, 3, 64, device=at[0]), Spec(calls.c_at, 2, at[1]), Tensor(2, 3, 64, device=at[2]),
            Tensor(2, 3, 64, dtype=FLOAT32, device=at[3]), ints(2, 3, device=at[4]), ints(2, 2, device=at[5]), ints(2, 3, 2, device=at[6]))
    with pytest.raises(ValueError, match="cuda:"):
        calls.m.logits(*args, None)
    assert not calls.made


def test_logits_refuses_other_shapes_and_another_current_device(calls):
    good = [Tensor(2, 3, 64), None, None, None, ints(2, 3), None, None, None]
    for i, bad in ((0, Tensor(2, 64)), (1, Spec(calls.c_at, 3, 0)), (2, Tensor(2, 3, 64, dtype=FP16)), (3, Tensor(2, 3, 64)),
                   (3, Tensor(2, 3, 64, dtype=FLOAT32, strides=(200, 64, 1))), (4, ints(2, 2)), (5, ints(2, 3)), (6, ints(2, 3, 1))):
        args = list(good)
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            calls.m.logits(*args)
    calls.now = 1
    with pytest.raises(ValueError, match="current device"):
        calls.m.logits(*good)
    assert not calls.made


def test_pages(calls):
    assert calls.m.extend(calls.pool(), calls.batch(), ints(3), ints(3), ints(20), Tensor(24, dtype=INT64), ints(3), None, None) == 0
    a = calls.made[0][1]
    assert a[3:5] == (3, 20) and a[5:8] == (16, 32, 48) and a[8:10] == (10, 10)
    assert calls.m.extend(calls.pool(), None, ints(3), None, None, None, None, None, None) == 0
    assert calls.made[1][1][4] == 1 << 30 and calls.made[1][1][5] is None
    assert calls.m.trim(calls.pool(), ints(3), None, -1, None, None) == 0 and calls.made[2][1][3:5] == (-1, 3)
    assert calls.m.trim(calls.pool(), None, None, 7, 2, None) == 0 and calls.made[3][1][3:5] == (7, 2)


@pytest.mark.parametrize("which", range(6))
def test_pages_refuse_tensors_of_two_devices(calls, which):
    at = [0] * 6
    at[which] = 1
    args = (calls.pool(at[0]), calls.batch(at[1]), ints(3, device=at[2]), ints(3, device=at[3]), ints(20, device=at[4]),
            Tensor(24, dtype=INT64, device=at[5]), None, None, None)
    with pytest.raises(ValueError, match="cuda:"):
        calls.m.extend(*args)
    assert not calls.made


def test_pages_refuse_other_shapes(calls):
    good = [calls.pool(), calls.batch(), ints(3), ints(3), ints(20), None, ints(3), None, None]
    for i, bad in ((2, ints(2)), (2, None), (2, Tensor(3, dtype=INT64)), (3, ints(2)), (4, ints(4, 5)), (6, ints(4)), (7, 21),
                   (3, ints(3, strides=(2,)))):
        args = list(good)
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            calls.m.extend(*args)
    with pytest.raises(ValueError):
        calls.m.trim(calls.pool(), None, None, -1, None, None)
    calls.now = 1
    with pytest.raises(ValueError, match="current device"):
        calls.m.trim(calls.pool(), ints(3), None, -1, None, None)
    assert not calls.made


# ------------------------------------------------------------ the entry points' own checks
@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_draft_tcgen05_gb300 as pkg
    L = pkg.lib()
    L.dflash_linear_run.argtypes = [P, P, I64, I64, P, I64, P, I64, P]
    L.dflash_logits_adjust.argtypes = [P, I64, I64, I32, I32, I64, I32, P, P, I64, P, I64, I64, P, I64, I64, P, P, P]
    L.dflash_pages_extend.argtypes = [P, P, P, I32, I32, P, P, P, I64, I32, P, P, P, P]
    L.dflash_pages_trim.argtypes = [P, P, P, I32, I32, P]
    return pkg, L


def refused(lib, status, word, code=1):
    assert status == code and word in lib[0].dflash_last_error(), (status, lib[0].dflash_last_error())


def test_linear_refusals(lib):
    pkg, L = lib
    h = P()

    def init(W=4096, bias=None, **k):
        cfg = pkg.dflash_linear_config(**{**dict(n=64, k=64, w_stride=64, dtype=0, out_dtype=0, activation=0), **k})
        return L.dflash_linear_init(ctypes.byref(cfg), W, bias, None, ctypes.byref(h))
    refused(lib, init(W=None), "NULL")
    refused(lib, init(W=4104), "aligned")
    refused(lib, init(w_stride=63), "W must")
    refused(lib, init(w_stride=68), "W must")
    refused(lib, init(bias=4097), "bias")
    refused(lib, init(activation=5), "activation")
    refused(lib, init(n=0), "n and k", 2)
    refused(lib, init(k=1 << 31), "n and k", 2)
    refused(lib, init(dtype=2), "dtype", 2)
    refused(lib, init(out_dtype=1), "out_dtype", 2)
    refused(lib, L.dflash_linear_run(None, 16, 64, 1, None, 0, 16, 64, None), "handle")
    assert L.dflash_linear_destroy(None) == 0


def test_logits_refusals(lib):
    pkg, L = lib

    def adjust(x=4096, batch=2, rows=2, vocab=64, dtype=0, rules=None, out=None, probs=None, best=64, draft=None, strides=(128, 64), outs=(128, 64)):
        return L.dflash_logits_adjust(x, *strides, batch, rows, vocab, dtype, None if rules is None else ctypes.addressof(rules),
                                      draft, 1, None, 0, 0, out, *outs, probs, best, None)
    refused(lib, adjust(dtype=2), "dtype", 2)
    refused(lib, adjust(batch=-1), "batch")
    refused(lib, adjust(vocab=0), "vocab")
    refused(lib, adjust(vocab=(1 << 30) + 1), "vocabulary", 2)
    refused(lib, adjust(best=None), "one of")
    refused(lib, adjust(x=None), "logits")
    refused(lib, adjust(x=4097), "aligned")
    refused(lib, adjust(probs=66), "aligned")
    refused(lib, adjust(strides=(-1, 64)), "strides")
    refused(lib, adjust(out=8192, outs=(128, 63)), "strides")
    refused(lib, adjust(out=4096, outs=(256, 64)), "strides")
    refused(lib, adjust(rules=pkg.dflash_logits_rules(tokens=64, token_cols=4, token_stride=4)), "lens")
    refused(lib, adjust(rules=pkg.dflash_logits_rules(tokens=64, lens=64, token_cols=4, token_stride=3)), "stride")
    refused(lib, adjust(rules=pkg.dflash_logits_rules(bias_ids=64, bias_count=4, bias_stride=4)), "biases")
    refused(lib, adjust(rules=pkg.dflash_logits_rules(temperature=66)), "aligned")
    assert adjust(batch=0, x=None, best=None) == 0


@pytest.mark.parametrize("kw", [dict(probs=4096, dtype=3), dict(probs=4600), dict(probs=4032, best=None), dict(best=4604),
                                dict(out=8192, probs=8700), dict(out=8192, best=8700), dict(probs=8192, best=9212),
                                dict(batch=1, rows=1, out=4222)])
def test_logits_refuse_outputs_that_overlap(lib, kw):
    """Logits at 4096 (2 x 2 x 64 values of 16 bits: to 4607), rows of out likewise, 1024 bytes of probs, 16 of best."""
    pkg, L = lib
    c = {**dict(batch=2, rows=2, dtype=0, out=None, probs=None, best=64), **kw}
    refused(lib, L.dflash_logits_adjust(4096, 128, 64, c["batch"], c["rows"], 64, c["dtype"], None, None, 1, None, 0, 0, c["out"],
                                        128, 64, c["probs"], c["best"], None), "overlap")


def test_pages_refusals(lib):
    pkg, L = lib

    def pool(**k):
        return pkg.dflash_page_pool(**{**dict(page_table=64, table_stride=8, lens=64, free_pages=64, counters=64, requests=4, cols=8,
                                              page_size=16, num_pages=32), **k})

    def extend(q, batch=2, tokens=8, rows=None, new=64, lens=None, table=None, stride=8, cols=8):
        return L.dflash_pages_extend(None if q is None else ctypes.addressof(q), rows, new, batch, tokens, 64, lens, table, stride, cols, None,
                                     None, None, None)
    refused(lib, extend(None), "pool")
    refused(lib, extend(pool(lens=None)), "given")
    refused(lib, extend(pool(counters=66)), "aligned")
    refused(lib, extend(pool(page_size=0)), "page_size")
    refused(lib, extend(pool(cols=(1 << 20) + 1)), "cols")
    refused(lib, extend(pool(cols=1 << 20, table_stride=1 << 20, page_size=4096)), "below 2^31")
    refused(lib, extend(pool(table_stride=7)), "table_stride")
    refused(lib, extend(pool(), batch=5), "batch")
    refused(lib, extend(pool(), batch=-1), "batch")
    refused(lib, extend(pool(), tokens=-1), "tokens")
    refused(lib, extend(pool(), new=None), "new_tokens")
    refused(lib, extend(pool(), table=128, cols=0), "table_cols")
    refused(lib, extend(pool(), table=128, stride=7), "table_stride")
    refused(lib, extend(pool(), rows=64, lens=64), "rows")
    refused(lib, extend(pool(), table=64, stride=9, cols=8), "stride")
    refused(lib, L.dflash_pages_trim(ctypes.addressof(pool()), None, None, -1, 5, None), "batch")
    assert L.dflash_pages_trim(ctypes.addressof(pool()), None, None, -1, 0, None) == 0
