"""The marshalling of the attention block's calls (csrc/paged_call.c), on the
CPU: a copy of the helper module with recording entry points and stand-ins for
tensors, which it knows only by their attributes."""
import ctypes
import importlib.util
import shutil

import pytest

P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
BF16, FP16, INT32, FLOAT32 = "bf16", "fp16", "int32", "float32"


class Tensor:
    def __init__(self, *shape, dtype=BF16, device=0, at=4096):
        self.dtype, self.shape, self.device, self.at = dtype, tuple(shape), device, at

    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s)

    def get_device(self):
        return self.device

    def data_ptr(self):
        return self.at

    def is_contiguous(self):
        return True


class Spec:
    def __init__(self, *spec):
        self.spec = spec


class Calls:
    """The module, with what its entry points were called with."""

    def __init__(self, path):
        spec = importlib.util.spec_from_file_location("_paged_call", path)
        self.m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(self.m)
        self.made, self.now, self.keep = [], 0, []
        at = []
        for name, args in (("norm_rope", [P, I64, I64] * 4 + [I32] * 5 + [P, P, P]),
                           ("append", [P, P, P, P, I64, I64, P, I64, I64, P, P, P, I64, I64, P, I64, I64, P]),
                           ("attend", [P, P, P, P, I64, I64, P, I64, I64, P, I32, I32, ctypes.c_float, P])):
            f = ctypes.CFUNCTYPE(ctypes.c_int, *args)(lambda *a, name=name: self.made.append((name, a)) or 0)
            self.keep.append(f)
            at.append(ctypes.cast(f, P).value)
        f = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: self.now)
        self.keep.append(f)
        self.m.setup(*at, ctypes.cast(f, P).value, lambda index: 1000 + index, INT32, FLOAT32, BF16, FP16)
        self.c = ctypes.create_string_buffer(512)  # stands for every C structure
        self.c_at = ctypes.addressof(self.c)

    def transform(self, device=-1, dtype=None):
        return Spec(self.c_at, dtype, 64 if dtype else 0, device)

    def objects(self, handle=0, cache=0, batch=0):
        shape = (16, 2, 64)
        return (Spec(self.c_at, BF16, BF16, 8, 2, 64, shape, handle), Spec(self.c_at, BF16, shape, cache), Spec(self.c_at, batch))


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    from speculative_decoding_draft_tcgen05_gb300 import build
    build.build()
    at = tmp_path_factory.mktemp("call") / "_paged_call.so"  # its own copy: the module's state is per file
    shutil.copy(build.CALL, at)
    return Calls(str(at))


@pytest.fixture(autouse=True)
def fresh(calls):
    calls.made.clear()
    calls.now = 0


def q(device=0, **k):
    return Tensor(4, 8, 64, device=device, **k)


def kv(device=0, **k):
    return Tensor(4, 2, 64, device=device, **k)


def test_calls_go_to_the_tensors_device(calls):
    calls.now = 1
    t = calls.transform(1, BF16)
    assert calls.m.norm_rope(q(1), kv(1), q(1), kv(1), t, Tensor(4, dtype=INT32, device=1), None) == 0
    h, c, b = calls.objects(1, 1, 1)
    assert calls.m.append(h, c, b, kv(1), kv(1), t, q(1), q(1), None, None) == 0
    assert calls.m.attend(h, c, b, q(1), q(1), Tensor(4, 8, dtype=FLOAT32, device=1), True, 0, None, None) == 0
    assert [n for n, _ in calls.made] == ["norm_rope", "append", "attend"]
    assert all(a[-1] == 1001 for _, a in calls.made)  # its current stream
    assert calls.m.norm_rope(q(1), None, q(1), None, calls.transform(), None, 77) == 0 and calls.made[-1][1][-1] == 77
    name, a = calls.made[2]
    assert a[4] == 512 and a[5] == 64 and a[10:12] == (1, 0) and a[12] == 0.125


@pytest.mark.parametrize("which", range(6))
def test_norm_rope_refuses_tensors_of_two_devices(calls, which):
    at = [0] * 6
    at[which] = 1
    args = (q(at[0]), kv(at[1]), q(at[2]), kv(at[3]), calls.transform(at[4], BF16), Tensor(4, dtype=INT32, device=at[5]), None)
    with pytest.raises(ValueError, match="cuda:"):
        calls.m.norm_rope(*args)
    assert not calls.made


def test_norm_rope_refuses_another_current_device(calls):
    for device, now in ((0, 1), (1, 0)):
        calls.now = now
        with pytest.raises(ValueError, match="current device"):
            calls.m.norm_rope(q(device), None, q(device), None, calls.transform(), None, None)
    assert not calls.made


@pytest.mark.parametrize("which", range(9))
def test_append_refuses_tensors_of_two_devices(calls, which):
    at = [0] * 9
    at[which] = 1
    args = (*calls.objects(*at[:3]), kv(at[3]), kv(at[4]), calls.transform(at[5], BF16), q(at[6]), q(at[7]),
            Tensor(4, dtype=INT32, device=at[8]), None)
    with pytest.raises(ValueError, match="cuda:"):
        calls.m.append(*args)
    assert not calls.made


@pytest.mark.parametrize("which", range(6))
def test_attend_refuses_tensors_of_two_devices(calls, which):
    at = [0] * 6
    at[which] = 1
    args = (*calls.objects(*at[:3]), q(at[3]), q(at[4]), Tensor(4, 8, dtype=FLOAT32, device=at[5]), True, 0, None, None)
    with pytest.raises(ValueError, match="cuda:"):
        calls.m.attend(*args)
    assert not calls.made


def test_host_tensors_are_refused(calls):
    for args in ((q(-1), None, q(), None), (q(), None, q(-1), None), (None, kv(-1), None, kv())):
        with pytest.raises(ValueError, match="CUDA tensor"):
            calls.m.norm_rope(*args, calls.transform(), None, None)
    assert not calls.made
