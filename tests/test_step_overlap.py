"""Outputs that share bytes with a call's other tensors are refused, slices of
one buffer that do not are told from them: csrc/spans.h against sets of bytes,
and the entry points' own checks, which come before any launch."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


@pytest.fixture(scope="module")
def spans(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("needs a C++ compiler")
    at = tmp_path_factory.mktemp("spans")
    (at / "spans.cpp").write_text("""#include "spans.h"
extern "C" int meets(const dfl::Rows *a, const dfl::Rows *b) { return dfl::meet(*a, *b); }
extern "C" int folds_over(const dfl::Rows *a) { return dfl::folds(*a); }
""")
    so = str(at / "spans.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "speculative_decoding_draft_tcgen05_gb300", "csrc"), str(at / "spans.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


class Rows(ctypes.Structure):
    _fields_ = [("at", P), ("width", I64), ("inner", I64), ("stride", I64), ("outer", I64), ("outer_stride", I64)]

    def bytes(self):
        return [self.at + i * self.outer_stride + j * self.stride + k
                for i in range(self.outer) for j in range(self.inner) for k in range(self.width)]


def test_rows_that_share_bytes(spans):
    r = random.Random(1)
    shared = passed = 0
    for _ in range(20000):
        a, b = (Rows(1000 + r.randint(0, 120), r.randint(1, 9), r.randint(1, 5), r.randint(0, 20), r.randint(1, 4), r.randint(0, 60))
                for _ in range(2))
        if r.random() < 0.7:
            b.stride, b.outer_stride = a.stride, a.outer_stride
        x, y = a.bytes(), b.bytes()
        assert spans.folds_over(ctypes.byref(a)) == (len(set(x)) < len(x))
        meet, got = not set(x).isdisjoint(y), spans.meets(ctypes.byref(a), ctypes.byref(b))
        same = (a.inner == 1 or b.inner == 1 or a.stride == b.stride) and (a.outer == 1 or b.outer == 1 or a.outer_stride == b.outer_stride)
        assert got == meet if same else got or not meet
        shared += meet
        passed += same and not meet and max(x) > min(y) and max(y) > min(x)
    assert shared > 5000 and passed > 200  # (slices that pass one another were among them)
    nothing = Rows(None, 8, 1, 0, 1, 0)
    assert not spans.meets(ctypes.byref(nothing), ctypes.byref(nothing))


@pytest.fixture(scope="module")
def lib():
    import speculative_decoding_draft_tcgen05_gb300 as pkg
    L = pkg.lib()
    L.dflash_logits_adjust.argtypes = [P, I64, I64, I32, I32, I64, I32, P, P, I64, P, I64, I64, P, I64, I64, P, P, P]
    L.dflash_pages_extend.argtypes = [P, P, P, I32, I32, P, P, P, I64, I32, P, P, P, P]
    L.dflash_pages_trim.argtypes = [P, P, P, I32, I32, P]
    return pkg, L


def refused(lib, status):
    assert status == 1 and "overlap" in lib[0].dflash_last_error(), (status, lib[0].dflash_last_error())


# Logits of 16 bits [2, 2, 64] at 4096, rows 128 bytes and sequences 256 bytes apart: to 4607.
@pytest.mark.parametrize("kw", [
    dict(out=4096 + 256),                               # the next sequence's place
    dict(out=4096 - 128), dict(out=4096 + 128),         # the next position's
    dict(out=4096 + 2), dict(out=4096 + 510),
    dict(out=65536, outs=(64, 64)),                     # sequences of out on one another
    dict(out=65536, outs=(96, 128)),
    dict(x=(64, 1024), outs=(96, 1024), out=4096 + 64),   # other strides, within the same bytes
], ids=str)
def test_logits_refuse_out_over_the_logits(lib, kw):
    xs, outs = kw.get("x", (128, 64)), kw.get("outs", (128, 64))
    refused(lib, lib[1].dflash_logits_adjust(4096, *xs, 2, 2, 64, 0, None, None, 1, None, 0, 0, kw["out"], *outs, None, None, None))


@pytest.mark.parametrize("which", ["draft", "mask", "tokens", "lens", "prompt_lens", "repetition", "presence", "frequency", "temperature",
                                   "bias_ids", "bias_values"])
@pytest.mark.parametrize("output", ["out", "probs", "argmax"])
def test_logits_refuse_outputs_over_inputs(lib, which, output):
    pkg, L = lib
    at = dict(out=1 << 16, probs=1 << 17, argmax=1 << 18)
    given = {output: at[output]}
    r = pkg.dflash_logits_rules(tokens=1 << 20, token_stride=4, token_cols=4, lens=(1 << 20) + 256, bias_ids=(1 << 20) + 512,
                                bias_values=(1 << 20) + 1024, bias_stride=4, bias_count=4)
    draft = mask = None
    if which == "draft":
        draft = at[output]
    elif which == "mask":
        mask = at[output]
    else:
        setattr(r, which, at[output])
    refused(lib, L.dflash_logits_adjust(4096, 128, 64, 2, 2, 64, 0, ctypes.addressof(r), draft, 1, mask, 4, 2, given.get("out"), 128, 64,
                                        given.get("probs"), given.get("argmax"), None))
