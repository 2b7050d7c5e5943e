"""The expert layers and 8-bit products on the GPU against the reference in 64
bits (stored forms and whole numbers bit for bit).

Tolerances, derived from the arithmetic (U = 2^-24, an FP32 rounding; S the sum
of the magnitudes that are added; h half a step of the output's type):
* a product: every one of the K products and sums of an output can be off by
  one rounding towards zero (2 U) of at most S, scales and joins by a few more:
  (K + 64) 2 U S;  4-bit weights with BF16 enter as 128 + q, at most 143, and
  136 times the row comes off: each block of 128 adds 256 numbers and a few sums
  whose partial sums are at most 279 s |a| summed: 320 2 U 279 sum(|a| s) more;
  the output's own rounding: h |y|, at least half its smallest step;
* the gate: silu has slope within +-1.1 and |silu(x)| <= |x|, exp and
  reciprocal are within 2^-21: 1.1 dx |u| + |silu(x)| du + dx du 1.1 + 2^-20 |y|;
* routing weights: exp of a difference d rounded once (|d| U) and exp itself
  (2 U), sums of at most 1024 such terms in 64 partial ones, two divisions:
  (2 max|d| + 64) U relative;
* the weighted sum: k products and sums: (k + 1) U S and the output's rounding.
"""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
import oracle
from oracle import moe_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _torch():
    import torch
    return torch


def _dtype(name):
    return getattr(_torch(), name)


def cuda(x):
    return _torch().from_numpy(np.ascontiguousarray(x)).cuda()


def to16(x, name):
    """float64/32 -> a device tensor of the 16-bit type and its exact values."""
    t = _torch().from_numpy(np.asarray(x, np.float32)).to(_dtype(name)).cuda()
    return t, t.double().cpu().numpy()


def host(t):
    return t.double().cpu().numpy()


def half_step(name):
    return float(_torch().finfo(_dtype(name)).eps) / 2


def least(name):
    """Half the smallest step of the type."""
    return 2.0 ** -25 if name == "float16" else 2.0 ** -134


def close(got, want, bound, what, name=None):
    """``name``: the type got was rounded to.  What rounds past FP16's largest
    value (65504 and half a step) is infinity."""
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= bound)
    if name == "float16":
        bad &= ~(np.isinf(got) & (got * want > 0) & (np.abs(want) + bound >= 65520.0))
    bad &= ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4],
                           np.broadcast_to(bound, got.shape)[bad][:4])


# ---------------------------------------------------------------------------
# 8-bit products
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("N,K", [(16, 128), (144, 640), (4096, 1024), (16384, 20480)])
def test_repack(N, K):
    say("repack", N, K)
    q = np.random.default_rng(0).integers(0, 256, (N, K)).astype(np.uint8)
    out = w4.alloc_w8a8_packed(K, N)
    w4.w8a8_repack(cuda(q), out)
    assert np.array_equal(out.view(_torch().uint8).cpu().numpy().reshape(-1), ref.repack8(q))


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,K", [(1, 128), (3, 384), (77, 1408), (5000, 256), (300001, 128)])
def test_quantize(T, K, name):
    torch = _torch()
    say("quantize", T, K, name)
    rng = np.random.default_rng(T)
    x = rng.standard_normal((T, K)) * np.exp(rng.uniform(-9, 6, (T, 1)))
    if T > 1:
        x[0] = 0.0
        x[1, ::7] = -x[1, ::7] * 3000.0
        x[2, 5], x[2, 130 % K] = np.inf, np.nan
    full, _ = to16(np.concatenate([x, x], 1)[:, :K + 24], name)
    t = full[:, 8:K + 8]                                    # strided rows, 16-byte aligned
    exact = host(t)
    q = torch.full((T, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((T, K // 128), -1.0, device="cuda")
    w4.w8a8_quantize(t, q, s)
    want_q, want_s = ref.quantise(exact.astype(np.float32))
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
def test_quantize_every_value(name):
    """Each 16-bit value beside a largest one of several sizes."""
    torch = _torch()
    say("quantize every value", name)
    bits = np.arange(65536, dtype=np.uint16).view(np.int16).reshape(-1, 64)
    v = torch.from_numpy(bits).view(_dtype(name))
    v = torch.where(v.float().isfinite(), v, torch.zeros_like(v))
    tops = torch.tensor([0.0, 1e-7, 1.0, 7.0, 448.0, 60000.0])
    x = torch.zeros((6, 1024, 128), dtype=_dtype(name))
    x[:, :, :64] = v
    x[:, :, 64] = tops.to(_dtype(name))[:, None]
    x = x.view(-1, 128).cuda()
    q = torch.empty((6144, 128), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((6144, 1), device="cuda")
    w4.w8a8_quantize(x, q, s)
    want_q, want_s = ref.quantise(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want_q)


def _e4m3(rng, shape):
    """Codes of finite values, of sizes that quantised rows have."""
    return ref.e4m3_code(rng.standard_normal(shape) * 100.0)


def _scales(rng, shape):
    return np.exp(rng.uniform(-3, 3, shape)).astype(np.float32)


def _dense(M, K, N, seed):
    rng = np.random.default_rng(seed)
    a, sa = _e4m3(rng, (M, K)), _scales(rng, (M, K // 128)) / 300.0
    b, sb = _e4m3(rng, (N, K)), _scales(rng, (-(-N // 128), K // 128)) / 300.0
    return a, sa, b, sb


def _run_dense(a, sa, b, sb, name, workspace=None, packed=None):
    torch = _torch()
    M, K, N = a.shape[0], a.shape[1], b.shape[0]
    if packed is None:
        packed = w4.alloc_w8a8_packed(K, N)
        w4.w8a8_repack(cuda(b), packed)
    room = torch.full((M + 3, N), 7.0, dtype=_dtype(name), device="cuda")
    ws = workspace if workspace is not None else w4.alloc_w8a8_workspace(M, K, N)
    w4.w8a8_gemm(cuda(a), cuda(sa), packed, cuda(sb), room[:M], ws)
    got = host(room)
    assert (got[M:] == 7.0).all()
    return got[:M]


def _dense_bound(a, sa, b, sb, name):
    x, w = ref.dequantise(a, sa), ref.weights8(b, sb).T
    y, S = x @ w, np.abs(x) @ np.abs(w)
    h = half_step(name)
    return y, (a.shape[1] + 64) * 2 * U * S * (1 + h) + h * np.abs(y) + least(name)


DENSE = [(1, 128, 16), (3, 256, 144), (16, 4096, 48), (17, 1408, 304), (33, 2048, 80),
         (48, 640, 528), (49, 1152, 144), (64, 2048, 272), (65, 3968, 400), (128, 2304, 128),
         (129, 1024, 656), (257, 384, 1040), (1100, 640, 272), (2300, 256, 528)]


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("M,K,N", DENSE)
def test_dense(M, K, N, name):
    say("dense", M, K, N, name, w4.w8a8_describe(M, K, N))
    case = _dense(M, K, N, M + K + N)
    got = _run_dense(*case, name)
    want, bound = _dense_bound(*case, name)
    close(got, want, bound, "dense", name)


def test_dense_is_deterministic_and_leaves_its_workspace_ready():
    torch = _torch()
    shapes = [(100, 4096, 272), (65, 8192, 144), (300, 2048, 128), (100, 4096, 272)]
    need = max(w4.w8a8_workspace_bytes(*s) for s in shapes)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = {}
    for M, K, N in shapes * 2:
        say("dense again", M, K, N)
        got = _run_dense(*_dense(M, K, N, 5), "float16", ws)
        assert np.array_equal(got, first.setdefault((M, K, N), got))
        assert not ws[:65536].any()
        want, bound = _dense_bound(*_dense(M, K, N, 5), "float16")
        close(got, want, bound, (M, K, N))


@pytest.mark.parametrize("M,K,N", [(5, 512, 48), (70, 2048, 144), (300, 512, 272)])
def test_dense_non_finite_and_extreme(M, K, N):
    """NaN stays in its row or column, overflow is infinity, zeros are zero."""
    say("dense non-finite", M, K, N)
    a, sa, b, sb = _dense(M, K, N, 1)
    sa[1, K // 128 - 1] = np.nan                             # a row that was not finite
    a[2, 77] = 0x7F                                          # a NaN code
    b[35, K - 1] = 0xFF
    a[3] = 0
    sa[4] = 1e30
    got = _run_dense(a, sa, b, sb, "float16")
    assert np.isnan(got[1]).all() and np.isnan(got[2]).all() and np.isnan(got[:, 35]).all()
    rest = np.delete(np.delete(got, 35, 1), [1, 2, 4], 0)
    assert np.isfinite(rest).all()
    assert (np.delete(got[3], 35) == 0).all()
    assert np.isinf(np.delete(got[4], 35)).all()


def test_dense_without_its_workspace_is_refused():
    torch = _torch()
    M, K, N = 100, 4096, 272
    assert w4.w8a8_workspace_bytes(M, K, N) > 0
    a, sa, b, sb = (cuda(x) for x in _dense(M, K, N, 0))
    c = torch.full((M, N), 3.0, dtype=torch.float16, device="cuda")
    with pytest.raises(w4.W4A16Error) as e:
        w4.w8a8_gemm(a, sa, b, sb, c)
    assert e.value.name == "W4A16_ERR_WORKSPACE"
    with pytest.raises(ValueError):
        w4.w8a8_gemm(a, sa, b, sb, c, torch.zeros(1000, dtype=torch.uint8, device="cuda"))
    assert (c == 3.0).all()


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def _check_route(x, bias, k, T=None, **kind):
    torch = _torch()
    T, E = x.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    call = dict(kind)
    softmax = call.pop("softmax", True)
    w4.moe_route(x, None if bias is None else cuda(bias.astype(np.float32)), ids, w,
                 score=w4.MOE_SOFTMAX if softmax else w4.MOE_SIGMOID, **call)
    exact = host(x)
    want_ids, want_w = ref.route(exact, bias, k, softmax=softmax, **call)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want_ids), np.argwhere(got != want_ids)[:4]
    finite = exact[np.isfinite(exact)]
    span = float(finite.max() - finite.min()) if finite.size else 0.0
    close(host(w), want_w, (2 * span + 64) * U * np.abs(want_w) + 1e-37, "weights")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 4, 2), (50, 8, 2), (33, 60, 4), (7, 64, 6),
                                   (130, 128, 8), (65, 160, 6), (41, 256, 8), (9, 384, 8),
                                   (5, 512, 10), (6, 1000, 32), (3, 1024, 1)])
@pytest.mark.parametrize("softmax", [True, False])
@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
def test_route(T, E, k, softmax, name):
    say("route", T, E, k, softmax, name)
    rng = np.random.default_rng(T * E + k)
    x = _torch().from_numpy(rng.standard_normal((T, E + 5)) * 2.0).to(_dtype(name)).cuda()
    bias = (rng.standard_normal(E) * 0.2).astype(np.float32).astype(np.float64)
    for b in (None, bias):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            # rows E + 5 apart, from an odd element on
            _check_route(x[:, 3:E + 3], b, k, softmax=softmax, renorm=renorm, scale=scale)


@pytest.mark.parametrize("E,groups,top", [(64, 8, 3), (256, 8, 4), (160, 8, 3), (384, 4, 2),
                                          (60, 4, 1), (128, 64, 9), (1024, 16, 16), (12, 12, 5)])
@pytest.mark.parametrize("best", [1, 2])
def test_route_groups(E, groups, top, best):
    say("route groups", E, groups, top, best)
    rng = np.random.default_rng(E + groups)
    x = cuda(rng.standard_normal((37, E)).astype(np.float32) * 1.5)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32).astype(np.float64)
    for softmax in (True, False):
        for b in (None, bias):
            _check_route(x, b, min(8, E), softmax=softmax, groups=groups, top_groups=top,
                         group_best=best)


def test_route_masked_tied_and_infinite():
    rng = np.random.default_rng(4)
    inf, nan = np.inf, np.nan
    x = rng.standard_normal((16, 48)).astype(np.float32)
    x[0] = -inf                                              # no expert at all
    x[1] = nan
    x[2, 3:] = -inf                                          # fewer than k
    x[3, ::2] = nan
    x[4] = 0.25                                              # all tied
    x[5, 7] = x[5, 31] = inf                                 # shared
    x[6, 7], x[6, 9] = inf, -inf
    x[7] = np.float32(-3.4028235e38)                         # the lowest value is a value
    x[8, :24] = np.float32(-3.4028235e38)
    x[9] = np.repeat(rng.standard_normal(12), 4)             # ties of four
    x[10] = 1e4 * x[10]
    bias = np.round(rng.standard_normal(48), 2).astype(np.float32).astype(np.float64)
    masked = bias.copy()
    masked[:40], masked[41] = -inf, nan
    for b in (None, bias, masked, np.zeros(48)):
        for softmax in (True, False):
            for kind in (dict(), dict(groups=6, top_groups=2, group_best=2),
                         dict(groups=6, top_groups=3, group_best=1), dict(renorm=False)):
                say("route masked", None if b is None else b[0], softmax, kind)
                _check_route(cuda(x), b, 6, softmax=softmax, **kind)


@pytest.mark.parametrize("name", ["float32", "float16"])
@pytest.mark.parametrize("T", [5, 4200])                     # 64 and 16 lanes a token
def test_route_zeros_of_both_signs_tie(T, name):
    say("route zeros", T, name)
    rng = np.random.default_rng(6)
    x = np.where(rng.random((T, 96)) < 0.5, -0.0, 0.0)
    x[:, ::7] = -1.0
    x = _torch().from_numpy(x).to(_dtype(name)).cuda()
    for kind in (dict(), dict(groups=8, top_groups=3), dict(groups=8, top_groups=3, group_best=2)):
        for softmax in (True, False):
            _check_route(x, None, 6, softmax=softmax, **kind)
            _check_route(x, np.full(96, -0.0), 6, softmax=softmax, **kind)


def test_route_near_ties_go_by_64_bits():
    """Scores a few FP32 roundings apart, where 32 bits would turn the order."""
    say("route near ties")
    rng = np.random.default_rng(5)
    x = (1.0 + rng.integers(0, 40, (200, 64)) * 2.0 ** -23).astype(np.float32)
    bias = (rng.integers(0, 3, 64) * 2.0 ** -24).astype(np.float32).astype(np.float64)
    for softmax in (True, False):
        _check_route(cuda(x), bias, 8, softmax=softmax)
        _check_route(cuda(x), None, 8, softmax=softmax)
        _check_route(cuda(x), None, 8, softmax=softmax, groups=8, top_groups=3, group_best=2)


@pytest.mark.parametrize("T,k,E", [(0, 2, 5), (1, 1, 1), (1, 8, 256), (40, 2, 8), (513, 8, 60),
                                   (1024, 1, 1024), (3000, 4, 3), (20001, 6, 64), (70000, 8, 384)])
def test_tables(T, k, E):
    torch = _torch()
    say("tables", T, k, E)
    rng = np.random.default_rng(T + E)
    for kind in range(4):
        ids = rng.integers(0, E, (T, k))
        if kind == 1:
            ids = rng.integers(-3, E + 4, (T, k))            # some of nobody
        elif kind == 2:
            ids = np.full((T, k), E - 1)                     # all of one
        elif kind == 3:
            ids = np.where(rng.random((T, k)) < 0.5, -2 ** 31, 2 ** 31 - 1)
        ids = ids.astype(np.int32)
        starts, order, where = w4.alloc_moe_tables(T, k, E)
        for t in (starts, order, where):
            t.fill_(-9)
        w4.moe_tables(cuda(ids), starts, order, where)
        if T * k > 50000:                                    # the reference loops over experts
            flat = np.where((ids.reshape(-1) < 0) | (ids.reshape(-1) >= E), E, ids.reshape(-1))
            o = np.argsort(flat, kind="stable").astype(np.int32)
            n = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])])
            wh = np.full(T * k, -1)
            wh[o[:n[E]]] = np.arange(n[E])
            o[n[E]:] = -1
            want = n, o, wh.reshape(T, k)
        else:
            want = ref.tables(ids, E)
        for got, w, what in zip((starts, order, where), want, ("starts", "order", "where")):
            assert np.array_equal(got.cpu().numpy(), w), (what, kind)


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def _weights(form, E, K, W, group, name, rng):
    """(packed, scales) on the device, the exact [E, K, W] and, of 4 bits, the
    scale of each."""
    torch = _torch()
    if form == 8:
        packed = w4.alloc_w8a8_packed(K, W, E)
        sb = _scales(rng, (E, -(-W // 128), K // 128)) / 300.0
        exact = np.empty((E, K, W))
        for e in range(E):
            q = _e4m3(rng, (W, K))
            w4.w8a8_repack(cuda(q), packed[e])
            exact[e] = ref.weights8(q, sb[e]).T
        return packed, cuda(sb), exact, None
    packed = torch.empty((E, K * W // 8), dtype=torch.int32, device="cuda")
    s, exact_s = to16(rng.uniform(0.005, 0.02, (E, K // group, W)), name)
    steps = np.repeat(exact_s, group, 1)
    exact = np.empty((E, K, W))
    for e in range(E):
        words = rng.integers(0, 2 ** 32, (K // 8, W), dtype=np.uint64).astype(np.uint32)
        w4.w4a16_repack(cuda(words.view(np.int32)), packed[e], K, W)
        codes = (words[:, None, :] >> (4 * np.arange(8, dtype=np.uint32))[None, :, None]) & 15
        exact[e] = (codes.reshape(K, W).astype(float) - 8) * steps[e]
    return packed, s, exact, steps


def _loads(kind, T, k, E, rng):
    """Ids [T, k]: experts with unlike, no, or all rows."""
    if kind == "one":
        return np.full((T, k), E // 2, np.int32)
    if kind == "elsewhere":
        return rng.integers(-1, 2 * E, (T, k)).astype(np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    p = np.exp(1.5 * rng.standard_normal(E))
    return rng.choice(E, (T, k), p=p / p.sum()).astype(np.int32)


def _run_experts(form, T, k, E, K, N, name, up, kind, group=128, seed=0):
    torch = _torch()
    rng = np.random.default_rng(seed + T + E + N)
    W = 2 * N if up else N
    packed, scales, exact_w, steps = _weights(form, E, K, W, group, name, rng)
    ids = _loads(kind, T, k, E, rng)
    starts, order, where = ref.tables(ids, E)
    rows = T * k
    a_rows = T if up else rows
    y = torch.full((rows + 2, N), 7.0, dtype=_dtype(name), device="cuda")
    idx = (cuda(order) if up else None, cuda(starts))
    act = w4.MOE_ACT_SILU_GATE if up else w4.MOE_ACT_NONE
    if form == 8:
        q, sa = _e4m3(rng, (a_rows, K)), _scales(rng, (a_rows, K // 128)) / 300.0
        A = ref.dequantise(q, sa)
        w4.w8a8_moe_gemm(cuda(q), cuda(sa), *idx, packed, scales, y[:rows], k, act)
    else:
        a, A = to16(rng.standard_normal((a_rows, K)), name)
        w4.w4a16_moe_gemm(a, *idx, packed, scales, y[:rows], k, group, act)
    got = host(y)
    assert (got[starts[E]:] == 7.0).all()
    x, S = ref.expert_rows(A, order if up else None, starts, exact_w, k, rows)
    n = starts[E]
    got, x, S = got[:n], x[:n], S[:n]
    h = half_step(name)
    d = (K + 64) * 2 * U * S
    if form == 4 and name == "bfloat16":
        more = ref.expert_rows(np.abs(A), order if up else None, starts, steps, k, rows)[0][:n]
        d = d + 320 * 2 * U * 279 * more
    if up:
        g, u, dg, du = x[:, :N], x[:, N:], d[:, :N], d[:, N:]
        s = ref.silu(g)
        y64 = s * u
        d = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(y64)
    else:
        y64 = x
    close(got, y64, d * (1 + h) + h * np.abs(y64) + least(name), (form, T, k, E, K, N, up),
          name)


EXPERTS = [
    (1, 1, 1, 128, 32, "skew"), (1, 2, 8, 256, 160, "skew"), (5, 2, 8, 1408, 96, "skew"),
    (24, 8, 60, 256, 96, "skew"), (9, 4, 3, 640, 352, "one"), (40, 2, 4, 512, 288, "elsewhere"),
    (70, 2, 5, 384, 160, "skew"), (130, 2, 4, 640, 416, "skew"), (333, 4, 8, 256, 544, "skew"),
    (600, 2, 3, 384, 288, "elsewhere"), (700, 3, 2, 256, 544, "skew"), (3, 2, 300, 256, 64, "skew"),
    (30, 2, 1024, 128, 32, "skew"), (50, 2, 4, 256, 96, "none"), (900, 2, 16, 256, 96, "one"),
    (2500, 1, 1, 256, 288, "skew"),
]


@pytest.mark.parametrize("up", [True, False])
@pytest.mark.parametrize("form,name", [(4, "float16"), (4, "bfloat16"), (8, "float16"),
                                       (8, "bfloat16")])
@pytest.mark.parametrize("T,k,E,K,N,kind", EXPERTS)
def test_experts(T, k, E, K, N, kind, form, name, up):
    say("experts", T, k, E, K, N, kind, form, name, up,
        w4.moe_gemm_describe(form, T * k, K, N, E, int(up)))
    _run_experts(form, T, k, E, K, N, name, up, kind)


@pytest.mark.parametrize("T,N", [(3, 48), (60, 80), (200, 176), (1200, 144)])
def test_experts_columns_of_16_and_long_groups(T, N):
    for up in (True, False):
        for name in ("float16", "bfloat16"):
            say("experts groups", T, N, up, name)
            _run_experts(4, T, 2, 2, 1536, N, name, up, "skew", group=384)
            _run_experts(4, T, 2, 2, 512, N, name, up, "skew", group=512)
    say("experts w8a8 columns", T, N)
    _run_experts(8, T, 2, 2, 512, N, "float16", False, "skew")


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("T", [2, 70, 300])                  # streamed, and both tiles
def test_experts_non_finite_rows_stay_alone(T, name):
    """Infinities and NaN in rows of A and in an expert's scales reach those
    rows and that expert's rows, and nothing else."""
    torch = _torch()
    rng = np.random.default_rng(T)
    k, E, K, N = 1, 2, 384, 288
    packed, scales, exact_w, _ = _weights(4, E, K, N, 128, name, rng)
    a, A = to16(rng.standard_normal((T, K)), name)
    ids = np.arange(T)[:, None].astype(np.int32) % 2
    starts, order, _ = ref.tables(ids, E)
    y = torch.empty((T, N), dtype=_dtype(name), device="cuda")
    say("experts non-finite", T, name, w4.moe_gemm_describe(4, T, K, N, E, 0))
    run = lambda: (w4.w4a16_moe_gemm(a, cuda(order), cuda(starts), packed, scales, y, k, 128),
                   host(y))[1]
    clean = run()
    assert np.isfinite(clean).all()
    a[0, 5], a[T - 1, K - 1] = float("nan"), float("inf")
    bad = np.isin(order, [0, T - 1])
    got = run()
    assert np.isnan(got[order == 0]).all() and not np.isfinite(got[bad]).any()
    assert np.array_equal(got[~bad], clean[~bad])
    a.copy_(torch.from_numpy(A))
    scales[1, 1, 7] = float("nan")                           # one column of one expert
    got = run()
    bad = np.zeros((T, N), bool)
    bad[starts[1]:, 7] = True
    assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], clean[~bad])


def test_experts_index_tensors_of_anything():
    """Orders and starts that hold nonsense: no row outside is touched, and
    rows whose entries are right are right."""
    torch = _torch()
    say("experts nonsense")
    rng = np.random.default_rng(0)
    T, k, E, K, N = 50, 2, 4, 256, 96
    packed, scales, exact_w, _ = _weights(4, E, K, N, 128, "float16", rng)
    a, A = to16(rng.standard_normal((T, K)), "float16")
    order = np.arange(100, dtype=np.int32)
    order[10], order[20], order[30] = -2 ** 31, 100, 2 ** 31 - 1
    starts = np.array([-50, 25, 60, 40, 2 ** 31 - 1], np.int32)
    y = torch.full((102, N), 7.0, dtype=torch.float16, device="cuda")
    w4.w4a16_moe_gemm(a, cuda(order), cuda(starts), packed, scales, y[:100], k, 128)
    got = host(y)
    assert (got[100:] == 7.0).all()
    src = np.where((order < 0) | (order >= 100), 0, order) // 2
    for p in range(25):                                      # expert 0: rows 0 .. 24
        want = A[src[p]] @ exact_w[0]
        S = np.abs(A[src[p]]) @ np.abs(exact_w[0])
        close(got[p], want, (K + 64) * 2 * U * S + 2.0 ** -11 * np.abs(want), p)


@pytest.mark.parametrize("T,k,N,rows", [(1, 1, 8, 1), (7, 2, 96, 14), (33, 8, 2048, 264),
                                        (40000, 2, 16, 80000), (5, 32, 4104, 20), (3, 2, 8, 0)])
@pytest.mark.parametrize("name", ["float16", "bfloat16"])
def test_combine(T, k, N, rows, name):
    torch = _torch()
    say("combine", T, k, N, rows, name)
    rng = np.random.default_rng(T + k)
    y, Y = to16(rng.standard_normal((rows, N)), name)
    where = rng.integers(-2, rows + 2, (T, k)).astype(np.int32)
    where[0] = -1
    weights = rng.uniform(0, 1, (T, k)).astype(np.float32)
    weights[where < 0] = np.nan                              # left out, whatever it is
    out = torch.full((T + 1, N), 7.0, dtype=_dtype(name), device="cuda")
    w4.moe_combine(y, cuda(where), cuda(weights), out[:T])
    got = host(out)
    assert (got[T:] == 7.0).all() and (got[0] == 0).all()
    live = (where >= 0) & (where < rows)
    P = np.concatenate([Y, np.zeros((1, N))])[np.where(live, where, rows)]
    w = np.where(live, weights, 0.0).astype(np.float64)[..., None]
    want, S = (w * P).sum(1), (w * np.abs(P)).sum(1)
    close(got[:T], want, (k + 1) * U * S * 2 + half_step(name) * np.abs(want) + least(name),
          "combine")


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

class Layer:
    """Routing, tables, both products and the sum of one layer of experts."""

    def __init__(self, form, T, k, E, K, N, name, seed=0):
        torch = _torch()
        rng = np.random.default_rng(seed)
        self.form, self.k, self.E, self.K, self.N = form, k, E, K, N
        self.w1, self.s1, self.x1, _ = _weights(form, E, K, 2 * N, 128, name, rng)
        self.w2, self.s2, self.x2, _ = _weights(form, E, N, K, 128, name, rng)
        dt = _dtype(name)
        self.x = torch.zeros((T, K), dtype=dt, device="cuda")
        self.logits = torch.zeros((T, E), dtype=dt, device="cuda")
        self.ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        self.weights = torch.zeros((T, k), device="cuda")
        self.starts, self.order, self.where = w4.alloc_moe_tables(T, k, E)
        self.h = torch.zeros((T * k, N), dtype=dt, device="cuda")
        self.y = torch.zeros((T * k, K), dtype=dt, device="cuda")
        self.out = torch.zeros((T, K), dtype=dt, device="cuda")
        self.q = [torch.zeros((n, c), dtype=torch.uint8, device="cuda")
                  for n, c in ((T, K), (T * k, N))]
        self.s = [torch.zeros((n, c // 128), device="cuda") for n, c in ((T, K), (T * k, N))]

    def run(self, stream=None):
        k = self.k
        w4.moe_route(self.logits, None, self.ids, self.weights, stream=stream)
        w4.moe_tables(self.ids, self.starts, self.order, self.where, stream=stream)
        if self.form == 8:
            w4.w8a8_quantize(self.x, self.q[0], self.s[0], stream=stream)
            w4.w8a8_moe_gemm(self.q[0], self.s[0], self.order, self.starts, self.w1, self.s1,
                             self.h, k, w4.MOE_ACT_SILU_GATE, stream=stream)
            w4.w8a8_quantize(self.h, self.q[1], self.s[1], stream=stream)
            w4.w8a8_moe_gemm(self.q[1], self.s[1], None, self.starts, self.w2, self.s2, self.y, k,
                             stream=stream)
        else:
            w4.w4a16_moe_gemm(self.x, self.order, self.starts, self.w1, self.s1, self.h, k, 128,
                              w4.MOE_ACT_SILU_GATE, stream=stream)
            w4.w4a16_moe_gemm(self.h, None, self.starts, self.w2, self.s2, self.y, k, 128,
                              stream=stream)
        w4.moe_combine(self.y, self.where, self.weights, self.out, stream=stream)

    def reference(self):
        """Token by token in 64 bits, rounded where a tensor is stored."""
        torch = _torch()
        x, logits = host(self.x), host(self.logits)
        if self.form == 8:
            x = ref.dequantise(*ref.quantise(x.astype(np.float32)))
        ids, weights = ref.route(logits, None, self.k)
        out = np.zeros(x.shape)
        for t in range(len(x)):
            for j, e in enumerate(ids[t]):
                z = x[t] @ self.x1[e]
                h = ref.silu(z[:self.N]) * z[self.N:]
                h = torch.from_numpy(h).to(self.h.dtype).double().numpy()
                if self.form == 8:
                    h = ref.dequantise(*ref.quantise(h[None].astype(np.float32)))[0]
                out[t] += weights[t, j] * (h @ self.x2[e])
        return out

    def check(self, what):
        got, want = host(self.out), self.reference()
        # codes next to a tie may fall the other way: a step of 2^-3 of a few
        # values; otherwise the roundings of the stored 16-bit tensors
        assert np.linalg.norm(got - want) <= 0.01 * np.linalg.norm(want), what


def _fill(layer, rng, scale=1.0):
    x = _torch().from_numpy(rng.standard_normal(tuple(layer.x.shape)) * scale)
    layer.x.copy_(x)
    layer.logits.copy_(_torch().from_numpy(2 * rng.standard_normal(tuple(layer.logits.shape))))


@pytest.mark.parametrize("form", [4, 8])
@pytest.mark.parametrize("T", [1, 9, 120, 700])
def test_layer(form, T):
    say("layer", form, T)
    layer = Layer(form, T, 2, 8, 512, 256, "float16" if T % 2 else "bfloat16")
    for i in range(2):
        _fill(layer, np.random.default_rng(i), 0.05)
        layer.run()
        layer.check((form, T, i))


@pytest.mark.parametrize("form", [4, 8])
def test_layer_replayed_from_a_graph(form):
    """Other tokens and other routing at every replay, eager work between."""
    torch = _torch()
    say("layer graph", form)
    layer = Layer(form, 21, 2, 6, 384, 256, "float16")
    _fill(layer, np.random.default_rng(0), 0.05)
    layer.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    for i in range(1, 5):
        _fill(layer, np.random.default_rng(i), 0.05)
        if i == 3:
            layer.logits[:, :5] = -float("inf")              # one expert for all, half the rows
        graph.replay()
        torch.cuda.synchronize()
        got = layer.out.clone()
        layer.out.zero_()
        layer.run()
        torch.cuda.synchronize()
        assert torch.equal(got, layer.out), i
        if i != 3:
            layer.check(i)


def test_layer_on_another_stream():
    torch = _torch()
    say("layer stream")
    layer = Layer(4, 40, 2, 6, 384, 256, "bfloat16")
    _fill(layer, np.random.default_rng(0), 0.05)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    layer.run(stream=side)
    side.synchronize()
    a = layer.out.clone()
    layer.run()
    assert torch.equal(a, layer.out)
    layer.check("stream")


def test_dense_replayed_from_a_graph():
    torch = _torch()
    say("dense graph")
    M, K, N = 100, 4096, 272
    a, sa, b, sb = (cuda(x) for x in _dense(M, K, N, 0))
    packed = w4.alloc_w8a8_packed(K, N)
    w4.w8a8_repack(b, packed)
    ws = w4.alloc_w8a8_workspace(M, K, N)
    assert ws is not None
    c = torch.zeros((M, N), dtype=torch.float16, device="cuda")
    x = torch.zeros((M, K), dtype=torch.float16, device="cuda")
    def step():
        w4.w8a8_quantize(x, a, sa)
        w4.w8a8_gemm(a, sa, packed, sb, c, ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        x.copy_(torch.randn((M, K), generator=torch.Generator().manual_seed(i)))
        graph.replay()
        torch.cuda.synchronize()
        got = c.clone()
        c.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, c) and got.abs().max() > 0


def test_two_graphs_share_a_workspace():
    """Products of unlike shapes that split K, captured over one workspace and
    replayed in turn."""
    torch = _torch()
    say("dense two graphs")
    shapes = [(100, 4096, 272), (60, 8192, 528), (33, 6144, 144)]
    ws = max((w4.alloc_w8a8_workspace(*s) for s in shapes), key=lambda w: w.numel())
    runs = []
    for i, (M, K, N) in enumerate(shapes):
        a, sa, b, sb = (cuda(x) for x in _dense(M, K, N, i))
        assert w4.w8a8_workspace_bytes(M, K, N) > 0
        packed = w4.alloc_w8a8_packed(K, N)
        w4.w8a8_repack(b, packed)
        c = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        call = lambda a=a, sa=sa, p=packed, sb=sb, c=c: w4.w8a8_gemm(a, sa, p, sb, c, ws)
        call()
        torch.cuda.synchronize()
        want = c.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, c, want, call))
    for i in range(9):
        graph, c, want, call = runs[i * i % 3 if i % 2 else i % 3]
        c.zero_()
        graph.replay() if i % 4 else call()
        torch.cuda.synchronize()
        assert torch.equal(c, want), i


def test_layers_on_two_streams_at_once():
    torch = _torch()
    say("two streams")
    layers = [Layer(8, 70, 2, 6, 384, 256, "bfloat16", 1), Layer(4, 150, 2, 8, 512, 256, "float16", 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for i, layer in enumerate(layers):
        _fill(layer, np.random.default_rng(i), 0.05)
        layer.run()
        want.append(layer.out.clone())
        layer.out.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for layer, stream in zip(layers, streams):
            layer.run(stream=stream)
    for layer, stream, w in zip(layers, streams, want):
        stream.synchronize()
        assert torch.equal(layer.out, w)


@pytest.mark.parametrize("T,k", [(700, 3), (9000, 4)])       # one launch, and three
def test_tables_of_most_experts_in_a_graph(T, k):
    torch = _torch()
    say("tables graph", T, k)
    E = w4.MOE_MAX_EXPERTS
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    starts, order, where = w4.alloc_moe_tables(T, k, E)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.moe_tables(ids, starts, order, where)
    for i in range(3):
        new = np.random.default_rng(i).integers(-2, E + 2, (T, k)).astype(np.int32)
        ids.copy_(_torch().from_numpy(new))
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((starts, order, where), ref.tables(new, E)):
            assert np.array_equal(got.cpu().numpy(), w), i


def test_binding_refusals_on_the_device():
    torch = _torch()
    x = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    q = torch.zeros((4, 256), dtype=torch.uint8, device="cuda")
    s = torch.zeros((4, 2), device="cuda")
    i = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        w4.w8a8_quantize(x, q[:3], s)
    with pytest.raises(ValueError):
        w4.w8a8_quantize(x.t(), q, s)
    with pytest.raises(w4.W4A16Error):
        w4.w8a8_quantize(x[:, :200], q, s)
    with pytest.raises(TypeError):
        w4.moe_route(q, None, i, s)
    with pytest.raises(ValueError):
        w4.moe_route(x, s[0], i, s)                          # a bias too short
    with pytest.raises(ValueError):
        w4.moe_tables(i, i.view(-1)[:3], i.view(-1)[:4], i)
    with pytest.raises(ValueError):
        w4.w4a16_moe_gemm(x, None, i.view(-1), i, x, torch.zeros((8, 16), dtype=torch.float16,
                                                                 device="cuda"), 1, 128)
    with pytest.raises(ValueError):
        w4.moe_combine(x, i, s.view(-1)[:7], x.clone())
