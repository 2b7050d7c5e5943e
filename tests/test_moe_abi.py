"""The C interface of the expert layers and 8-bit products on the CPU:
exports, sizes, plans, and every refusal before anything touches a device."""

from __future__ import annotations

import ctypes
import os
import re

import pytest

import weight_only_int4_gemm_amd as w4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

OK, NULL, SHAPE, GROUP, ALIGN, WORKSPACE, DEVICE, EPILOGUE, DTYPE = 0, -1, -2, -3, -4, -5, -7, -8, -9

# Fake, 16-byte aligned addresses far apart: the checks return before any of
# them is dereferenced or handed to the runtime.
A = [0x100000000000 + i * 0x10000000000 for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    return w4.load()


@pytest.fixture
def no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("accepted calls with fake addresses: without a device only")


@pytest.mark.parametrize("header,names", [("w8a8.h", w4.W8A8_EXPORTED_SYMBOLS),
                                          ("w4a16_moe.h", w4.MOE_EXPORTED_SYMBOLS)])
def test_header_binding_and_library_agree(lib, header, names):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b([a-z0-9_]+)\s*\([^)]*\)\s*;", text))) == sorted(names)
    for name in names:
        assert isinstance(getattr(lib, name), ctypes._CFuncPtr) and callable(getattr(w4, name))
    for name in re.findall(r"\b(MOE_[A-Z0-9_]+)\s*=", text):
        assert int(re.search(name + r"\s*=\s*(\d+)", text).group(1)) == getattr(w4, name)
    for name in re.findall(r"#define (MOE_[A-Z0-9_]+)\s+\d", text):
        assert int(re.search(name + r"\s+(\d+)", text).group(1)) == getattr(w4, name)
    assert w4.w8a8_layout_version() == 1


def _no(call, base, expect, **change):
    assert call(*{**base, **change}.values()) == expect, change


REPACK = dict(B=A[0], Bpacked=A[1], K=256, N=48, stream=None)
QUANT = dict(X=A[0], x_row=256, Xq=A[1], Xs=A[2], T=4, K=256, dtype=0, stream=None)
DENSE = dict(A=A[0], As=A[1], Bpacked=A[2], Bs=A[3], C=A[4], M=4, K=256, N=48, dtype=0,
             workspace=None, stream=None)
ROUTE = dict(logits=A[0], row=64, kind=2, bias=A[1], ids=A[2], weights=A[3], T=4, E=64, k=8,
             score=0, groups=8, top_groups=4, group_best=2, renorm=1, scale=1.0, stream=None)
TABLES = dict(ids=A[0], starts=A[1], order=A[2], where=A[3], T=8, k=2, E=16, stream=None)
INT4 = dict(A=A[0], a_rows=8, order=A[1], k=2, starts=A[2], Bpacked=A[3], scales=A[4], C=A[5],
            rows=16, K=256, N=48, group=128, E=4, activation=1, dtype=0, stream=None)
FP8 = dict(A=A[0], As=A[6], a_rows=8, order=A[1], k=2, starts=A[2], Bpacked=A[3], Bs=A[4], C=A[5],
           rows=16, K=256, N=64, E=4, activation=1, dtype=0, stream=None)
COMBINE = dict(Y=A[0], rows=16, where=A[1], weights=A[2], out=A[3], T=8, k=2, N=48, dtype=0,
               stream=None)


def test_accepted_calls_reach_the_device(lib, no_device):
    for call, base in ((lib.w8a8_repack, REPACK), (lib.w8a8_quantize, QUANT),
                       (lib.w8a8_gemm, DENSE), (lib.moe_route, ROUTE), (lib.moe_tables, TABLES),
                       (lib.w4a16_moe_gemm, INT4), (lib.w8a8_moe_gemm, FP8),
                       (lib.moe_combine, COMBINE)):
        assert call(*base.values()) == DEVICE


def test_repack_refusals(lib):
    assert w4.w8a8_packed_bytes(4096, 11008) == 4096 * 11008
    for K, N in ((0, 16), (128, 0), (64, 16), (128, 8), (-128, 16)):
        assert w4.w8a8_packed_bytes(K, N) == 0
        _no(lib.w8a8_repack, REPACK, SHAPE, K=K, N=N)
    _no(lib.w8a8_repack, REPACK, NULL, B=None)
    _no(lib.w8a8_repack, REPACK, NULL, Bpacked=None)
    _no(lib.w8a8_repack, REPACK, ALIGN, B=A[0] + 8)
    _no(lib.w8a8_repack, REPACK, ALIGN, Bpacked=A[1] + 8)
    _no(lib.w8a8_repack, REPACK, SHAPE, Bpacked=A[0] + 256 * 48 - 16)
    _no(lib.w8a8_repack, REPACK, SHAPE, K=128 << 20, N=16 << 20)      # no launch takes it


def test_quantize_refusals(lib):
    f = lib.w8a8_quantize
    for k in ("X", "Xq", "Xs"):
        _no(f, QUANT, NULL, **{k: None})
        _no(f, QUANT, ALIGN, **{k: QUANT[k] + 8})
    for bad in (dict(T=-1), dict(K=0), dict(K=192), dict(x_row=248), dict(x_row=-256),
                dict(T=(1 << 24) + 1)):
        _no(f, QUANT, SHAPE, **bad)
    _no(f, QUANT, ALIGN, x_row=260)
    _no(f, QUANT, DTYPE, dtype=2)
    _no(f, QUANT, SHAPE, Xq=A[0] + 16)
    _no(f, QUANT, SHAPE, Xs=A[1] + 1008)
    _no(f, QUANT, OK, T=0, X=None, Xq=None, Xs=None)


def test_dense_refusals(lib):
    f = lib.w8a8_gemm
    for k in ("A", "As", "Bpacked", "Bs", "C"):
        _no(f, DENSE, NULL, **{k: None})
        _no(f, DENSE, ALIGN, **{k: DENSE[k] + 8})
    _no(f, DENSE, ALIGN, workspace=A[9] + 4)
    for bad in (dict(M=-1), dict(M=(1 << 24) + 1), dict(K=0), dict(K=200), dict(N=-16), dict(N=24)):
        _no(f, DENSE, SHAPE, **bad)
    _no(f, DENSE, DTYPE, dtype=-1)
    for k, n in (("A", 4 * 256), ("As", 4 * 8), ("Bpacked", 256 * 48), ("Bs", 8)):
        _no(f, DENSE, SHAPE, C=DENSE[k] + n - 16 if n > 16 else DENSE[k])
    for empty in (dict(M=0), dict(N=0)):
        _no(f, DENSE, OK, A=None, As=None, Bpacked=None, Bs=None, C=None, **empty)
    assert w4.w8a8_workspace_bytes(4, 200, 48) == 0
    assert w4.w8a8_workspace_bytes(0, 256, 48) == 0


def test_route_refusals(lib):
    f = lib.moe_route
    for k in ("logits", "ids", "weights"):
        _no(f, ROUTE, NULL, **{k: None})
        _no(f, ROUTE, ALIGN, **{k: ROUTE[k] + 2})
    _no(f, ROUTE, ALIGN, bias=A[1] + 2)
    _no(f, ROUTE, ALIGN, logits=A[0] + 1, kind=0)
    _no(f, ROUTE, DTYPE, kind=3)
    for bad in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(k=5, E=4, groups=1,
                top_groups=1), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=7),
                dict(groups=65, E=65, row=65), dict(groups=128, E=128, row=128),
                dict(top_groups=0), dict(top_groups=9), dict(group_best=0), dict(group_best=3),
                dict(row=63)):
        _no(f, ROUTE, SHAPE, **bad)
    _no(f, ROUTE, SHAPE, ids=A[3] + 124)
    _no(f, ROUTE, SHAPE, weights=A[0] + 64 * 16 - 4)
    _no(f, ROUTE, SHAPE, ids=A[1] + 252)
    _no(f, ROUTE, OK, T=0, logits=None, ids=None, weights=None)


def test_tables_refusals(lib):
    f = lib.moe_tables
    for k in ("ids", "starts", "order", "where"):
        _no(f, TABLES, NULL, **{k: None})
        _no(f, TABLES, ALIGN, **{k: TABLES[k] + 2})
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(E=1025), dict(T=1 << 24)):
        _no(f, TABLES, SHAPE, **bad)
    for k in ("starts", "order", "where"):
        _no(f, TABLES, SHAPE, **{k: A[0] + 60})
    _no(f, TABLES, SHAPE, order=A[1] + 64)
    _no(f, TABLES, NULL, T=0, starts=None)


def test_experts_refusals(lib):
    for f, base, scales in ((lib.w4a16_moe_gemm, INT4, "scales"), (lib.w8a8_moe_gemm, FP8, "Bs")):
        for k in ("A", "starts", "Bpacked", scales, "C") + (("As",) if "As" in base else ()):
            _no(f, base, NULL, **{k: None})
            _no(f, base, ALIGN, **{k: base[k] + (2 if k == "starts" else 8)})
        _no(f, base, ALIGN, order=A[1] + 2)
        for bad in (dict(rows=-1), dict(rows=(1 << 24) + 1), dict(K=0), dict(K=192), dict(N=-32),
                    dict(N=24), dict(E=0), dict(E=1025), dict(k=0), dict(a_rows=0),
                    dict(N=1 << 30), dict(order=None)):  # 8 rows of A for 16
            _no(f, base, SHAPE, **bad)
        _no(f, base, DTYPE, dtype=2)
        _no(f, base, EPILOGUE, activation=2)
        for k, n in (("A", 2048), ("order", 64), ("starts", 20), ("Bpacked", 4 * 128 * 48),
                     (scales, 32)):
            _no(f, base, SHAPE, C=base[k] + n // 32 * 16)
        for empty in (dict(rows=0), dict(N=0)):
            _no(f, base, OK, A=None, starts=None, Bpacked=None, C=None, **{scales: None}, **empty)
    for group in (0, -128, 64, 384):
        _no(lib.w4a16_moe_gemm, INT4, GROUP, group=group)
    _no(lib.w8a8_moe_gemm, FP8, SHAPE, N=48)            # with the gate: multiples of 32
    # the last expert's weights count
    _no(lib.w4a16_moe_gemm, INT4, SHAPE, C=A[3] + 4 * 256 * 96 // 2 - 16)
    _no(lib.w8a8_moe_gemm, FP8, SHAPE, C=A[3] + 4 * 256 * 128 - 16)


def test_combine_refusals(lib):
    f = lib.moe_combine
    for k in ("Y", "where", "weights", "out"):
        _no(f, COMBINE, NULL, **{k: None})
        _no(f, COMBINE, ALIGN, **{k: COMBINE[k] + 2})
    for bad in (dict(T=-1), dict(k=0), dict(k=33), dict(N=-8), dict(N=12),
                dict(N=(1 << 24) + 8), dict(N=(1 << 31) - 8), dict(rows=-1)):
        _no(f, COMBINE, SHAPE, **bad)
    _no(f, COMBINE, DTYPE, dtype=2)
    _no(f, COMBINE, SHAPE, out=A[0] + 16 * 48 * 2 - 16)
    _no(f, COMBINE, SHAPE, out=A[1] + 48)
    _no(f, COMBINE, OK, T=0, Y=None, where=None, weights=None, out=None)


def _fields(text):
    return {k: v for k, v in re.findall(r"(\w+)=(\S+)", text)}


def test_plans_cover_every_row_and_column():
    """Tiles of any plan: enough for the most row tiles that routing can make."""
    for rows in (1, 15, 16, 17, 100, 1000, 4097, 65536):
        for E in (1, 8, 60, 256):
            for form, act, N in ((4, 0, 4096), (4, 1, 1408), (8, 1, 1440), (8, 0, 144)):
                d = _fields(w4.moe_gemm_describe(form, rows, 512, N, E, act, 256))
                tm, tn = map(int, d["tile"].split("x"))
                gm, gn = map(int, d["grid"].split("x"))
                assert gn == -(-N // tn)
                used = min(rows, E)
                # as many experts as can have one row past a whole tile
                spread = min(used, rows // 1)
                left, tiles = rows, 0
                for e in range(spread):
                    take = 1 if e < spread - 1 else left
                    tiles += -(-take // tm)
                    left -= take
                assert gm >= tiles and gm >= -(-rows // tm)
                assert d["splits"] == "1" and d["workspace"] == "0"


def test_dense_plans():
    for M in (1, 16, 17, 100, 512, 4096):
        for K, N in ((4096, 4096), (11008, 4096), (8192, 28672), (128, 16), (28672, 144)):
            d = _fields(w4.w8a8_describe(M, K, N, 256))
            tm, tn = map(int, d["tile"].split("x"))
            gm, gn = map(int, d["grid"].split("x"))
            splits = int(d["splits"])
            assert gm == -(-M // tm) and gn == -(-N // tn)
            assert 1 <= splits <= max(1, K // 128)
            assert (splits > 1) == (int(d["workspace"]) > 0)
            if splits > 1:
                assert gm * gn <= 16384
                assert int(d["workspace"]) >= 65536 + gm * gn * splits * tm * tn * 4


def test_describe_refusals():
    import weight_only_int4_gemm_amd as w4
    for call in (lambda: w4.w8a8_describe(0, 128, 16, 256), lambda: w4.w8a8_describe(4, 100, 16, 256),
                 lambda: w4.moe_gemm_describe(5, 4, 128, 16, 2, 0, 256),
                 lambda: w4.moe_gemm_describe(8, 4, 128, 16, 2, 1, 256),
                 lambda: w4.moe_gemm_describe(4, 4, 128, 16, 0, 0, 256),
                 lambda: w4.moe_gemm_describe(4, 4, 128, 16, 2, 3, 256),
                 # 2^32 threads and more
                 lambda: w4.moe_gemm_describe(4, 1 << 24, 128, 1 << 22, 4, 1, 256),
                 lambda: w4.moe_gemm_describe(8, 1 << 24, 128, 1 << 24, 4, 0, 256),
                 lambda: w4.w8a8_describe(1 << 24, 128, 1 << 24, 256)):
        with pytest.raises(w4.W4A16Error):
            call()


def test_binding_refusals_without_a_device():
    """Host tensors, wrong types and shapes are Python errors."""
    import torch
    x = torch.zeros((4, 256), dtype=torch.float16)
    q = torch.zeros((4, 256), dtype=torch.uint8)
    s = torch.zeros((4, 2))
    i = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.w8a8_quantize(x, q, s)
    with pytest.raises(TypeError):
        w4.w8a8_quantize(x.float(), q, s)
    with pytest.raises(ValueError):
        w4.w8a8_gemm(q, s, q, s, torch.zeros((5, 16), dtype=torch.float16))
    with pytest.raises(TypeError):
        w4.w8a8_repack(x, q)
    with pytest.raises(ValueError):
        w4.moe_route(torch.zeros((4, 8)), None, i, s)
    with pytest.raises(ValueError):
        w4.moe_tables(i, i[0], i, i)
    with pytest.raises(ValueError):
        w4.moe_combine(x, i, s, x[:, :128].contiguous())
    with pytest.raises(ValueError):
        w4.alloc_w8a8_packed(100, 16)
