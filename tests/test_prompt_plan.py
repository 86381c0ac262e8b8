"""The launch arithmetic of the prompt and chunk attention kernels
(csrc/prompt_plan.h) on the CPU, for the SM counts of a GPU: what a call lays
into its workspace fits what the workspace query asks for."""
import ctypes
import os
import random
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "medusa_tree_speculative_heads_b200", "csrc")
SOURCE = """
#include "prompt_plan.h"
using namespace medusa;
extern "C" void plan(int sms, int tc, int B, int N, int max_new, int max_prefix, int Hq, int Hkv, long* out) {
    const PromptPlan p = prompt_plan(sms, tc != 0, B, N, max_new, max_prefix, Hq, Hkv);
    out[0] = p.T;
    out[1] = p.splits;
    out[2] = p.tiles;
    out[3] = p.table;
}
extern "C" size_t used(long rows, int D) { return split_bytes(rows, D); }
extern "C" size_t asked(int sms, int N, int Hq, int D) { return split_bytes(split_rows(sms, N, Hq), D); }
"""
LAYOUTS = [(32, 8), (64, 8), (64, 1), (4, 4), (5, 1), (6, 2), (14, 2), (33, 1), (1, 1), (36, 12)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("prompt_plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-O1", "-fPIC", "-shared", "-I", CSRC,
                           str(src), "-o", str(so)])
    L = ctypes.CDLL(str(so))
    i32, i64, sz = ctypes.c_int, ctypes.c_long, ctypes.c_size_t
    L.plan.argtypes, L.plan.restype = [i32] * 8 + [ctypes.POINTER(i64)], None
    L.used.argtypes, L.used.restype = [i64, i32], sz
    L.asked.argtypes, L.asked.restype = [i32, i32, i32, i32], sz
    return L


def _plan(lib, *args):
    out = (ctypes.c_long * 4)()
    lib.plan(*args, out)
    return dict(zip(("T", "splits", "tiles", "table"), out))


def _fits(lib, sms, tc, B, N, max_new, max_prefix, Hq, Hkv, D):
    p = _plan(lib, sms, tc, B, N, max_new, max_prefix, Hq, Hkv)
    what = (sms, tc, B, N, max_new, max_prefix, Hq, Hkv, D, p)
    assert 1 <= p["splits"] <= 64, what
    if p["splits"] > 1:
        assert lib.used(p["splits"] * N * Hq, D) <= lib.asked(sms, N, Hq, D), what
        assert not p["table"], what  # (it would lie in the same workspace)
    return p


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,N,max_new,max_prefix,Hq,Hkv", [
    (1, 127, 64, 32768, 32, 8), (1, 67, 60, 20000, 32, 8), (2, 255, 64, 32768, 32, 8), (1, 191, 64, 32768, 32, 8),
    (2, 255, 64, 8192, 32, 8), (4, 319, 64, 8192, 32, 8), (1, 6399, 6144, 0, 1, 1), (1, 500, 256, 20000, 8, 8)])
def test_rows_of_no_sequence_fit_the_workspace(lib, B, N, max_new, max_prefix, Hq, Hkv, D):
    """More rows than B * max_new fill: the tiles do not cover them, the
    partials of split keys are laid out for them all the same."""
    _fits(lib, 148, 1, B, N, max_new, max_prefix, Hq, Hkv, D)
    _fits(lib, 148, 0, B, N, max_new, max_prefix, Hq, Hkv, D)


def test_such_calls_still_split_their_keys(lib):
    assert _plan(lib, 148, 1, 1, 127, 64, 32768, 32, 8)["splits"] == 37888 // (127 * 32)


@pytest.mark.parametrize("sms", [1, 16, 132, 148])
@pytest.mark.parametrize("tc", [0, 1])
def test_layouts_fit_the_workspace(lib, sms, tc):
    rng = random.Random(100 * sms + tc)
    for Hq, Hkv in LAYOUTS:
        T = 2 * (128 // (Hq // Hkv)) if tc else max(64 // (Hq // Hkv), 1)
        lengths = sorted({1, 2, 16, T - 1, T, T + 1, 2 * T - 1, 3 * T - 1, 7 * T + 3, 25 * T - 1} - {0})
        for B in (1, 2, 3, 17):
            for N in lengths + [rng.randint(1, 40 * T) for _ in range(6)]:
                for max_new in {n for n in lengths if n <= N} | {N, rng.randint(1, N)}:
                    for max_prefix in (0, 400, 8192, 131072, 1 << 30):
                        _fits(lib, sms, tc, B, N, max_new, max_prefix, Hq, Hkv, 128)


@pytest.mark.parametrize("tc", [0, 1])
def test_covered_rows_split_to_fill_the_gpu(lib, tc):
    """Calls whose rows all lie in tiles are split as the SMs ask, not by the
    workspace."""
    for Hq, Hkv in LAYOUTS:
        for B in (1, 3, 8):
            for n in (1, 5, 33, 64, 100, 257, 1024):
                for max_prefix in (0, 3000, 40000):
                    p = _plan(lib, 148, tc, B, B * n, n, max_prefix, Hq, Hkv)
                    chunks = -(-(max_prefix + n) // (128 if tc else 64))
                    fill = (1 if tc else 2) * 148 // (p["tiles"] * Hkv)
                    assert p["splits"] == max(1, min(fill, chunks // (8 if tc else 1), 64)), (Hq, Hkv, B, n, p)


def test_a_workspace_serves_calls_of_fewer_rows(lib):
    last = 0
    for n in range(0, 2000, 7):
        a = lib.asked(148, n, 32, 128)
        assert a >= last
        last = a
