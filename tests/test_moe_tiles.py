"""The cases of tests/test_gpu_moe_tiles.py on the CPU: each gets the kernel it
is for, and every compiled variant has a case."""

from __future__ import annotations

import os
import re

import weight_only_int4_gemm_amd as w4
from tests.test_gpu_moe_tiles import CUS, DENSE, EXPERTS, planned
from weight_only_int4_gemm_amd import build as wbuild


def test_cases_get_their_kernels():
    for M, K, N, shape, splits, tile in DENSE:
        assert planned(w4.w8a8_describe(M, K, N, CUS)) == (tile, shape, splits), (M, K, N)
    for form, gate, rows, K, N, E, shape, tile in EXPERTS:
        text = w4.moe_gemm_describe(form, rows, K, N, E, gate, CUS)
        assert planned(text) == (tile, shape, 1), (form, gate, rows, K, N, E, text)


def _compiled():
    """(form, tile, shape, gate) of every kernel that product_launch.hpp lists."""
    text = open(os.path.join(wbuild.CSRC, "product_launch.hpp")).read().replace("\\\n", " ")
    out = set()
    for kind, form, items in re.findall(r"#define W4A16_(STREAM|TILE)_(F8|I4)\(X\)(.*)", text):
        form = 8 if form == "F8" else 4
        for entry in re.findall(r"X\(([\d, ]+)\)", items):
            a, b, c, d = map(int, entry.split(","))
            if kind == "STREAM":
                out |= {(form, 0, (a, b, c, d), gate) for gate in range(2 if b % 2 == 0 else 1)}
            else:                        # depth 4: the stages
                out |= {(form, 1, (a, b, c, 4), gate) for gate in range(2 if d else 1)}
    return out


def test_every_compiled_variant_has_a_case():
    have = {(8, tile, shape, 0) for _, _, _, shape, _, tile in DENSE}
    have |= {(form, tile, shape, gate) for form, gate, _, _, _, _, shape, tile in EXPERTS}
    compiled = _compiled()
    assert len(compiled) == 21
    assert compiled == have, (compiled - have, have - compiled)
    # the tiles of matrix products in every number of K ranges that a plan gives them
    assert {(s, n) for _, _, _, s, n, t in DENSE if t} == {
        ((2, 1, 4, 4), 1), ((2, 1, 4, 4), 2), ((2, 1, 4, 4), 4), ((2, 1, 4, 4), 8),
        ((4, 1, 4, 4), 1), ((4, 1, 4, 4), 2), ((4, 1, 4, 4), 4), ((4, 1, 4, 4), 8),
        ((4, 2, 4, 4), 1), ((4, 2, 4, 4), 2), ((4, 2, 4, 4), 4), ((4, 2, 4, 4), 8),
        ((8, 2, 4, 4), 1), ((8, 2, 4, 4), 2), ((8, 2, 4, 4), 4),
        ((8, 4, 4, 4), 1), ((8, 4, 4, 4), 2), ((8, 4, 4, 4), 4)}
