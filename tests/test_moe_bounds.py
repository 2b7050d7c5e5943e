"""Bounds of moe_tables on the CPU: how it divides its choices
(csrc/tables_plan.hpp), compiled for the host."""

from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from weight_only_int4_gemm_amd import build as wbuild

COMPILER = next((c for c in map(shutil.which, ("g++", "c++", "clang++")) if c), None)
ONE_LAUNCH = 16384          # choices up to which no counts are kept
MOST = 1 << 24              # choices of a call

# For every E of 1 .. experts and each n: 0, or what is wrong and where.
HARNESS = """
#include "tables_plan.hpp"
using namespace w4a16;
extern "C" int one_launch() { return kTablesOneLaunch; }
extern "C" int chunk(int n, int E) { return table_chunk(n, E); }
extern "C" int groups(int n, int chunk) { return table_groups(n, chunk); }
extern "C" int first_bad(int lo, int hi, int step, int experts, int* bad_n, int* bad_E) {
  for (int n = lo; n <= hi; n += step)
    for (int E = 1; E <= experts; ++E) {
      const int c = table_chunk(n, E), g = table_groups(n, c);
      int what = 0;
      if (c % 1024 || c <= 0) what = 1;                        // threads take whole rounds
      if (g < 1 || g > 256) what = 2;
      if ((int64_t)g * c < n || (int64_t)(g - 1) * c >= (n ? n : 1)) what = 3;  // covers n
      if (n > kTablesOneLaunch && (int64_t)g * E > n) what = 4;  // counts fit in order
      if (what) { *bad_n = n; *bad_E = E; return what; }
    }
  return 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if COMPILER is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("tables_plan")
    src, lib = d / "harness.cpp", d / "harness.so"
    src.write_text(HARNESS)
    subprocess.run([COMPILER, "-O2", "-std=c++17", "-shared", "-fPIC", "-I", wbuild.CSRC,
                    "-o", str(lib), str(src)], check=True)
    return ctypes.CDLL(os.fspath(lib))


@pytest.mark.parametrize("n,E", [(16385, 964), (16385, 1024), (16640, 1000), (36000, 1024),
                                 (262143, 1024), (17407, 1024)])
def test_counts_of_a_short_last_chunk_fit(plan, n, E):
    c = plan.chunk(n, E)
    # in chunks of 1024 they would not
    assert -(-n // 1024) * E > n
    assert plan.groups(n, c) * E <= n


def test_every_size_is_covered_and_its_counts_fit(plan):
    assert plan.one_launch() == ONE_LAUNCH
    n, E = ctypes.c_int(), ctypes.c_int()
    for lo, hi, step in ((0, ONE_LAUNCH, 97), (ONE_LAUNCH, ONE_LAUNCH + 6000, 1),
                         (ONE_LAUNCH, 1 << 19, 127), (1 << 18, (1 << 18) + 2100, 1),
                         (1 << 19, MOST, 65521), (MOST - 3, MOST, 1)):
        what = plan.first_bad(lo, hi, step, 1024, ctypes.byref(n), ctypes.byref(E))
        assert what == 0, (what, n.value, E.value)


def test_sizes_whose_counts_fitted_are_divided_as_before(plan):
    for n, E in ((16385, 8), (24588, 128), (131072, 128), (131072, 1024), (120006, 64),
                 (560000, 384), (MOST, 1024), (1, 1), (0, 5), (16384, 1024)):
        chunk = 1024
        while chunk * 256 < n:
            chunk *= 2
        assert plan.chunk(n, E) == chunk, (n, E)
