"""How attention cuts its work, on the CPU: the host side of csrc/paged.cuh
against Python integers, at sizes whose sums do not fit 32 bits."""
import os
import shutil
import subprocess

import pytest

PROGRAM = r"""
#include <stdio.h>
#include "paged.cuh"
using namespace dfl;
int main()
{
    int n, len, group, causal, window, R, U, C;
    while (scanf("%d %d %d %d %d %d %d %d", &n, &len, &group, &causal, &window, &R, &U, &C) == 8) {
        AttendParams p = {};
        p.group = group;
        p.by_group = FastDiv(group);
        p.causal = causal;
        p.window = window;
        const PagedSeq s = {0, n, len};
        const PagedCut cut = {R, U, C};
        const int tiles = paged_row_tiles(p, s, R);
        const PagedItem last = paged_item(p, s, tiles > 0 ? tiles - 1 : 0, cut);
        printf("%d %d %d %d %d %lld\n", tiles, last.lo, last.hi, last.u0, last.units, static_cast<long long>(paged_cost(p, s, cut)));
    }
    return 0;
}
"""

FEW, MANY = (8, 64, 5), (256, 128, 4)
CASES = [
    (1, 1, 1, 1, 0, *FEW), (8, 2049, 4, 1, 0, *FEW), (300, 300, 4, 1, 0, *MANY), (1100, 3275, 8, 1, 1024, *MANY),
    (40, 7, 3, 1, 0, *FEW), (200, 700, 5, 0, 100, *MANY),
    (1 << 20, 1 << 20, 64, 0, 0, *MANY),            # 2^18 row tiles of 2^13 units
    (1 << 20, 1 << 20, 64, 1, 0, *FEW),             # 2^23 of 2^13 on average
    (1 << 21, (1 << 31) - 4096, 64, 0, 0, *FEW),
    (1 << 24, (1 << 31) - 4096, 127, 0, 1 << 30, *MANY),  # rows close to 2^31
]


def item(n, length, group, causal, window, R, U, C, rt):
    r0, r1 = rt * R, min(n * group, rt * R + R)
    base = length - n
    hi = min(length, max(0, base + (r1 - 1) // group + 1)) if causal else length
    lo = max(0, base + r0 // group - window + 1) if window else 0
    if lo >= hi:
        lo = hi = 0
    u0 = lo // U
    return lo, hi, u0, max(1, -(-hi // U) - u0)


def cost(n, length, group, causal, window, R, U, C):
    """The same sum, tile by tile where they are few, else by tokens' runs of equal bounds (R a multiple of group or not)."""
    tiles = -(-n * group // R)
    if tiles <= 1 << 16:
        return sum(item(n, length, group, causal, window, R, U, C, t)[3] + C for t in range(tiles))
    import numpy as np
    total = 0
    for t0 in range(0, tiles, 1 << 20):
        rt = np.arange(t0, min(tiles, t0 + (1 << 20)), dtype=np.int64)
        r0, r1 = rt * R, np.minimum(n * group, rt * R + R)
        base = length - n
        hi = np.minimum(length, np.maximum(0, base + (r1 - 1) // group + 1)) if causal else np.full_like(rt, length)
        lo = np.maximum(0, base + r0 // group - window + 1) if window else np.zeros_like(rt)
        gone = lo >= hi
        lo, hi = np.where(gone, 0, lo), np.where(gone, 0, hi)
        total += int((np.maximum(1, -(-hi // U) - lo // U) + C).sum())
    return total


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from speculative_decoding_draft_tcgen05_gb300 import build
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("needs nvcc")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cu").write_text(PROGRAM)
    subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, str(at / "plan.cu"), "-o", str(at / "plan")], check=True)
    return str(at / "plan")


def test_costs_and_bounds(program):
    text = "\n".join(" ".join(map(str, c)) for c in CASES)
    got = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
    assert any(cost(*c) > 1 << 31 for c in CASES)
    for c, line in zip(CASES, got):
        tiles = -(-c[0] * c[2] // c[5])
        assert [int(x) for x in line.split()] == [tiles, *item(*c, tiles - 1), cost(*c)], c
