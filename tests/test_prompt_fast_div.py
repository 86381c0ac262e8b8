"""Division by a tile's token or head count as the attention kernels do it
(csrc/prompt_plan.h: a multiplication and a shift) on the CPU: exact for every
dividend below 2^31."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "medusa_tree_speculative_heads_b200", "csrc")
SOURCE = """
#include "prompt_plan.h"
extern "C" void divide(int T, const int* x, int* q, long n) {
    const medusa::FastDiv d = medusa::fast_div(T);
    for (long i = 0; i < n; ++i) q[i] = medusa::div_by(x[i], d);
}
"""


@pytest.fixture(scope="module")
def divide(tmp_path_factory):
    d = tmp_path_factory.mktemp("fast_div")
    src, so = d / "div.cpp", d / "div.so"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-O2", "-fPIC", "-shared", "-I", CSRC,
                           str(src), "-o", str(so)])
    f = ctypes.CDLL(str(so)).divide
    f.argtypes, f.restype = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_long], None

    def run(T, x):
        x = np.ascontiguousarray(x, dtype=np.int32)
        q = np.empty_like(x)
        f(T, x.ctypes.data, q.ctypes.data, x.size)
        return q
    return run


def test_every_divisor_is_exact(divide):
    """At multiples of the divisor and one below, where a quotient changes:
    the first and last of the range and 2^16 between; and at the powers of 2."""
    rng = np.random.default_rng(5)
    top = 2 ** 31 - 1
    for T in range(1, 257):
        k = np.concatenate([np.arange(1000), rng.integers(0, top // T + 1, 1 << 16), top // T - np.arange(1000)])
        x = np.concatenate([k * T, k * T - 1, k * T + T - 1, 2 ** np.arange(31), 2 ** np.arange(31) - 1, [top]])
        x = x[(x >= 0) & (x <= top)]
        assert np.array_equal(divide(T, x), x // T), T


@pytest.mark.parametrize("T", [1, 3, 7, 64, 85, 256])
def test_long_runs(divide, T):
    for first in (0, 2 ** 24 - 4096, 2 ** 30 - 4096, 2 ** 31 - (1 << 20)):
        x = np.arange(first, first + (1 << 20), dtype=np.int64)
        assert np.array_equal(divide(T, x), x // T)
