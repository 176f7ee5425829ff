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


# A pool of 4 requests and 8 columns, everything 4096 bytes apart.
POOL = dict(page_table=1 << 16, table_stride=10, lens=(1 << 16) + 4096, free_pages=(1 << 16) + 8192, counters=(1 << 16) + 12288,
            requests=4, cols=8, page_size=16, num_pages=32)
OUT = dict(cu=1 << 20, lens=(1 << 20) + 4096, table=(1 << 20) + 8192, positions=(1 << 20) + 12288, slots=(1 << 20) + 16384,
           granted=(1 << 20) + 20480)


def extend(lib, rows=None, new=1 << 19, stride=8, pool={}, **out):
    o = {**dict.fromkeys(OUT), **out}
    q = lib[0].dflash_page_pool(**{**POOL, **pool})
    return lib[1].dflash_pages_extend(ctypes.addressof(q), rows, new, 3, 8, o["cu"], o["lens"], o["table"], stride, 8, o["positions"],
                                      o["slots"], o["granted"], None)


@pytest.mark.parametrize("name", OUT)
def test_pages_refuse_outputs_over_the_pool_inputs_and_one_another(lib, name):
    last = dict(cu=12, lens=8, table=8 * 4 * 2 + 28, positions=28, slots=56, granted=8)[name]
    for base, size in ((POOL["lens"], 16), (POOL["page_table"], 10 * 4 * 3 + 32), (POOL["free_pages"], 128), (POOL["counters"], 8), (1 << 19, 12)):
        ends = (base - last // 8 * 8, base + (size - 4) // 8 * 8)
        for at in (*ends, base) if (base, name) not in ((POOL["lens"], "lens"), (POOL["page_table"], "table")) else ends:
            refused(lib, extend(lib, **{name: at}))
    for other in OUT:
        if other != name:
            refused(lib, extend(lib, **{**OUT, name: OUT[other]}))


def test_pages_refuse_inputs_over_the_pool(lib):
    for base in (POOL["lens"], POOL["page_table"], POOL["free_pages"], POOL["counters"]):
        refused(lib, extend(lib, rows=base))
        refused(lib, extend(lib, new=base + 4))
        q = lib[0].dflash_page_pool(**POOL)
        for rows, counts in ((base, None), (1 << 19, base), (None, base + 4)):
            refused(lib, lib[1].dflash_pages_trim(ctypes.addressof(q), rows, counts, -1, 3, None))
    refused(lib, extend(lib, rows=1 << 18, new=POOL["lens"]))
    refused(lib, extend(lib, pool=dict(lens=POOL["free_pages"] + 124)))
    refused(lib, extend(lib, pool=dict(counters=POOL["page_table"] + 32 + 40 * 3 - 4)))


def test_pages_refuse_a_view_of_the_pools_lengths_or_table_from_another_place(lib):
    refused(lib, extend(lib, lens=POOL["lens"] + 4))
    refused(lib, extend(lib, table=POOL["page_table"] + 40, stride=10))
    refused(lib, extend(lib, table=POOL["page_table"] + 4, stride=10))
