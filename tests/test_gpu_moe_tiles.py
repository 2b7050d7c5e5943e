"""Every compiled variant of the product kernels (csrc/product_launch.hpp) with
ragged rows, K blocks that end anywhere in the loop, and columns that end inside
a workgroup's; each case asserts the kernel and the K ranges that it is for.
tests/test_moe_tiles.py checks on the CPU that no variant is left out.

The reference is the definition in 64 bits, on the device: one matrix product
an expert, of codes looked up in oracle/moe_ref.py's table.

Tolerances (U = 2^-24, an FP32 rounding; S the sum of the magnitudes that are
added; h half a step of the output's type):
* a block of 128 is summed by matrix instructions, 128 additions each off by at
  most one rounding towards zero of the block's S; the K / 128 blocks are then
  added one by one, and at most 8 K ranges; their scales are a few roundings
  more: (128 + K / 128 + 64) 2 U S;
* 4-bit weights with BF16 enter as 128 + q, at most 143, and 136 times the row
  comes off: 256 numbers and a few sums a block, whose partial sums are at most
  279 s |a| summed: 320 2 U 279 sum(|a| s) more;
* the gate: the exponent x log2(e) has two roundings (the constant's and the
  product's), which the exponential turns into 2 |x| U; exponential, sum,
  reciprocal and two products at most 8 U: (2 |x| + 8) U |y|.  Below x = -87.3
  the reciprocal is below 2^-126 and may be 0: |x| exp(x) |u| <= 2^-118 |u|.
  With dx, du off already: 1.1 dx |u| + |silu(x)| du + 1.1 dx du (silu's slope
  is within +-1.1);
* the output's own rounding: h |y|, at least half its smallest step.
"""

from __future__ import annotations

import re

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import moe_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CUS = 256

# M, K, N, (row blocks, column blocks, waves, depth), K ranges, tile kernel
DENSE = [
    (1, 640, 80, (1, 1, 8, 4), 1, 0), (16, 1408, 272, (1, 1, 8, 4), 1, 0),
    (13, 896, 12304, (1, 2, 4, 4), 1, 0), (17, 1408, 80, (2, 1, 8, 3), 1, 0),
    (31, 2944, 144, (2, 1, 8, 3), 1, 0),
    (33, 128, 16, (2, 1, 4, 4), 1, 1), (45, 384, 1040, (2, 1, 4, 4), 1, 1),
    (100, 1152, 144, (2, 1, 4, 4), 1, 1), (20, 3840, 16, (2, 1, 4, 4), 2, 1),
    (19, 7552, 16, (2, 1, 4, 4), 4, 1), (23, 29696, 16, (2, 1, 4, 4), 8, 1),
    (8197, 128, 16, (4, 1, 4, 4), 1, 1), (8321, 384, 16, (4, 1, 4, 4), 1, 1),
    (8364, 2560, 16, (4, 1, 4, 4), 1, 1), (4304, 6528, 16, (4, 1, 4, 4), 2, 1),
    (100, 11008, 4096, (4, 1, 4, 4), 2, 1), (2093, 26240, 16, (4, 1, 4, 4), 4, 1),
    (2167, 50048, 16, (4, 1, 4, 4), 8, 1),
    (135, 256, 16432, (4, 2, 4, 4), 1, 1), (202, 384, 12416, (4, 2, 4, 4), 1, 1),
    (5507, 2176, 144, (4, 2, 4, 4), 1, 1), (8804, 7680, 80, (4, 2, 4, 4), 2, 1),
    (4221, 14208, 80, (4, 2, 4, 4), 4, 1), (2213, 49920, 80, (4, 2, 4, 4), 8, 1),
    (5963, 384, 6544, (8, 2, 4, 4), 1, 1), (8752, 1920, 672, (8, 2, 4, 4), 1, 1),
    (8524, 5888, 208, (8, 2, 4, 4), 1, 1), (8214, 16384, 80, (8, 2, 4, 4), 2, 1),
    (4428, 40448, 80, (8, 2, 4, 4), 4, 1),
    (7239, 256, 13296, (8, 4, 4, 4), 1, 1), (6314, 384, 9840, (8, 4, 4, 4), 1, 1),
    (6551, 1664, 1824, (8, 4, 4, 4), 1, 1), (2822, 13952, 1424, (8, 4, 4, 4), 2, 1),
    (8369, 24960, 224, (8, 4, 4, 4), 4, 1),
]

# form, gate, rows, K, N, experts, shape, tile kernel
EXPERTS = [
    (8, 0, 9, 640, 160, 5, (1, 2, 4, 4), 0), (8, 1, 21, 1408, 96, 8, (1, 2, 4, 4), 0),
    (8, 0, 61, 384, 176, 5, (2, 2, 4, 4), 1), (8, 1, 61, 640, 160, 5, (2, 2, 4, 4), 1),
    (8, 0, 5167, 2688, 48, 4, (2, 2, 4, 4), 1), (8, 1, 2533, 2560, 64, 2, (2, 2, 4, 4), 1),
    (8, 0, 5522, 128, 912, 5, (4, 2, 4, 4), 1), (8, 1, 5627, 128, 480, 13, (4, 2, 4, 4), 1),
    (8, 0, 5217, 384, 400, 13, (4, 2, 4, 4), 1), (8, 1, 7258, 384, 160, 13, (4, 2, 4, 4), 1),
    (8, 0, 8478, 1920, 144, 13, (4, 2, 4, 4), 1), (8, 1, 8972, 1280, 96, 1, (4, 2, 4, 4), 1),
    (8, 0, 8795, 2432, 1040, 3, (8, 4, 4, 4), 1), (8, 1, 6583, 384, 3680, 4, (8, 4, 4, 4), 1),
    (8, 0, 5606, 2944, 1584, 2, (8, 4, 4, 4), 1), (8, 1, 7021, 3200, 608, 3, (8, 4, 4, 4), 1),
    (4, 0, 9, 640, 144, 5, (1, 2, 8, 3), 0), (4, 1, 9, 640, 144, 5, (1, 2, 8, 3), 0),
    (4, 0, 59, 2176, 2064, 16, (1, 4, 4, 3), 0), (4, 1, 59, 1408, 1040, 16, (1, 4, 4, 3), 0),
    (4, 0, 61, 384, 176, 5, (2, 2, 4, 4), 1), (4, 1, 61, 640, 144, 5, (2, 2, 4, 4), 1),
    (4, 0, 5028, 2560, 80, 4, (2, 2, 4, 4), 1), (4, 1, 5662, 3200, 48, 2, (2, 2, 4, 4), 1),
    (4, 0, 7984, 256, 4016, 1, (4, 4, 4, 4), 1), (4, 1, 7568, 128, 4608, 5, (4, 4, 4, 4), 1),
    (4, 0, 5959, 384, 3824, 2, (4, 4, 4, 4), 1), (4, 1, 8860, 384, 1232, 1, (4, 4, 4, 4), 1),
    (4, 0, 8539, 3712, 400, 4, (4, 4, 4, 4), 1), (4, 1, 6274, 2048, 336, 8, (4, 4, 4, 4), 1),
]


def planned(text):
    """(tile kernel, shape, K ranges) of a description."""
    m = re.match(r"product_(tile|stream)_kernel<([\d,]+)>.* splits=(\d+)", text)
    return int(m[1] == "tile"), tuple(map(int, m[2].split(","))), int(m[3])


def _assert_plan(text, describe, tile, shape, splits=1):
    import torch
    assert planned(text) == (tile, shape, splits), text
    if torch.cuda.get_device_properties(0).multi_processor_count == CUS:
        assert describe() == text


# ---------------------------------------------------------------------------
# inputs and the reference, on the device
# ---------------------------------------------------------------------------

def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, g):
    import torch
    return torch.randn(shape, device="cuda", generator=g, dtype=torch.float32)


def _codes(shape, g):
    import torch
    return (_randn(shape, g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(shape, g):
    return (_randn(shape, g)).exp() / 300


def _value(codes):
    import torch
    return torch.from_numpy(ref.e4m3_value(np.arange(256))).cuda()[codes.long()]


def _rows8(q, s):
    return _value(q) * s.double().repeat_interleave(128, 1)


def _weights8(q, s):
    """Codes [N][K] -> [K][N]."""
    s = s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)
    return (_value(q) * s).t().contiguous()


def _int4(words, s, group):
    """(values, scales) [K][N] of words [K/8][N] and scales [K/group][N]."""
    import torch
    shift = 4 * torch.arange(8, device="cuda", dtype=torch.int32)
    q = ((words[:, None, :] >> shift[None, :, None]) & 15).reshape(-1, words.shape[1])
    steps = s.double().repeat_interleave(group, 0)
    return (q.double() - 8) * steps, steps


def _close(got, want, bound, name, what):
    import torch
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    if name == "float16":                # past the largest value, 65504 and half a step
        bad &= ~(got.isinf() & (got * want > 0) & (want.abs() + bound >= 65520.0))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(),
                           want[bad][:4].tolist(), bound[bad][:4].tolist())


def _rounding(want, d, name):
    import torch
    h = float(torch.finfo(getattr(torch, name)).eps) / 2
    return d * (1 + h) + h * want.abs() + (2.0 ** -25 if name == "float16" else 2.0 ** -134)


def _sums(K):
    return (128 + K // 128 + 64) * 2 * U


def _gated(x, dx, N):
    """(y, bound) of the gate half times the up half."""
    import torch
    g, u, dg, du = x[:, :N], x[:, N:], dx[:, :N], dx[:, N:]
    s = g / (1 + torch.exp(-g))
    y = s * u
    d = (1.1 * dg * u.abs() + s.abs() * du + 1.1 * dg * du + (2 * g.abs() + 8) * U * y.abs()
         + 2.0 ** -118 * u.abs())
    return y, d


# ---------------------------------------------------------------------------
# matrix products
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,K,N,shape,splits,tile", DENSE)
def test_dense_variant(M, K, N, shape, splits, tile):
    import torch
    name = "bfloat16" if (M + K // 128) % 2 else "float16"
    say("dense variant", M, K, N, name, shape, splits)
    _assert_plan(w4.w8a8_describe(M, K, N, CUS), lambda: w4.w8a8_describe(M, K, N), tile, shape,
                 splits)
    g = _gen(M + K + N)
    a, sa = _codes((M, K), g), _scales((M, K // 128), g)
    b, sb = _codes((N, K), g), _scales((-(-N // 128), K // 128), g)
    packed = w4.alloc_w8a8_packed(K, N)
    w4.w8a8_repack(b, packed)
    c = torch.full((M + 3, N), 7.0, dtype=getattr(torch, name), device="cuda")
    ws = w4.alloc_w8a8_workspace(M, K, N)
    for _ in range(2):                   # the second call finds the workspace as the first left it
        c[:M] = float("nan")
        w4.w8a8_gemm(a, sa, packed, sb, c[:M], ws)
        assert (c[M:] == 7.0).all()
        first = c.clone() if _ == 0 else first
        assert torch.equal(first, c)
    x, w = _rows8(a, sa), _weights8(b, sb)
    want = x @ w
    S = x.abs() @ w.abs()
    _close(c[:M], want, _rounding(want, _sums(K) * S, name), name, (M, K, N))


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def _starts(rows, E, rng):
    """Unlike loads, one expert without rows where there are several, the last
    rows (one or two) of nobody where there are many."""
    p = np.exp(0.3 * rng.standard_normal(E))
    if E > 2:
        p[E // 2] = 0
    n = np.bincount(rng.choice(E, rows - (2 if rows > 100 else 0), p=p / p.sum()), minlength=E)
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


class Case:
    """Operands of one product on the device, and its reference."""

    def __init__(self, form, gate, rows, K, N, E, name, group=128, seed=0):
        import torch
        rng, g = np.random.default_rng(seed + rows + E), _gen(seed + rows + K + N)
        self.form, self.gate, self.rows, self.K, self.N, self.E = form, gate, rows, K, N, E
        self.name, self.group, W = name, group, N * (2 if gate else 1)
        self.starts = _starts(rows, E, rng)
        self.k = 2 if gate else 1        # gated: gathered from the tokens
        self.a_rows = -(-rows // self.k)
        self.order = rng.permutation(rows).astype(np.int32) if gate else None
        if form == 8:
            self.a, self.sa = _codes((self.a_rows, K), g), _scales((self.a_rows, K // 128), g)
            self.b = _codes((E, W, K), g)
            self.s = _scales((E, -(-W // 128), K // 128), g)
            self.packed = w4.alloc_w8a8_packed(K, W, E)
            for e in range(E):
                w4.w8a8_repack(self.b[e], self.packed[e])
        else:
            dt = getattr(torch, name)
            self.a = _randn((self.a_rows, K), g).to(dt)
            self.s = (torch.rand((E, K // group, W), device="cuda", generator=g) * 0.015
                      + 0.005).to(dt)
            self.b = torch.randint(-2 ** 31, 2 ** 31, (E, K // 8, W), device="cuda", generator=g,
                                   dtype=torch.int64).to(torch.int32)
            self.packed = torch.empty((E, K * W // 8), dtype=torch.int32, device="cuda")
            for e in range(E):
                w4.w4a16_repack(self.b[e], self.packed[e], K, W)
        self.y = torch.full((rows + 2, N), 7.0, dtype=getattr(torch, name), device="cuda")

    def run(self):
        import torch
        self.y.fill_(7.0)
        act = w4.MOE_ACT_SILU_GATE if self.gate else w4.MOE_ACT_NONE
        order = None if self.order is None else torch.from_numpy(self.order).cuda()
        starts = torch.from_numpy(self.starts).cuda()
        if self.form == 8:
            w4.w8a8_moe_gemm(self.a, self.sa, order, starts, self.packed, self.s,
                             self.y[:self.rows], self.k, act)
        else:
            w4.w4a16_moe_gemm(self.a, order, starts, self.packed, self.s, self.y[:self.rows],
                              self.k, self.group, act)
        return self.y.clone()

    def check(self):
        import torch
        y = self.run()
        assert (y[self.starts[self.E]:] == 7.0).all()
        x = _rows8(self.a, self.sa) if self.form == 8 else self.a.double()
        for e in range(self.E):
            lo, hi = int(self.starts[e]), int(self.starts[e + 1])
            if lo == hi:
                continue
            at = np.arange(lo, hi) if self.order is None else self.order[lo:hi] // self.k
            r = x[torch.from_numpy(at).cuda().long()]
            if self.form == 8:
                w, steps = _weights8(self.b[e], self.s[e]), None
            else:
                w, steps = _int4(self.b[e], self.s[e], self.group)
            want = r @ w
            d = _sums(self.K) * (r.abs() @ w.abs())
            if self.form == 4 and self.name == "bfloat16":
                d = d + 320 * 2 * U * 279 * (r.abs() @ steps)
            if self.gate:
                want, d = _gated(want, d, self.N)
            _close(y[lo:hi], want, _rounding(want, d, self.name), self.name, (e, lo, hi))


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("form,gate,rows,K,N,E,shape,tile", EXPERTS)
def test_experts_variant(form, gate, rows, K, N, E, shape, tile, name):
    say("experts variant", form, gate, rows, K, N, E, name, shape)
    _assert_plan(w4.moe_gemm_describe(form, rows, K, N, E, gate, CUS),
                 lambda: w4.moe_gemm_describe(form, rows, K, N, E, gate), tile, shape)
    Case(form, gate, rows, K, N, E, name).check()


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("gate,rows,K,N,E", [(0, 8539, 3712, 400, 4), (1, 6274, 2048, 336, 8)])
def test_large_4_bit_tiles_with_one_group(gate, rows, K, N, E, name):
    say("experts one group", gate, rows, K, N, E, name)
    assert planned(w4.moe_gemm_describe(4, rows, K, N, E, gate, CUS))[:2] == (1, (4, 4, 4, 4))
    Case(4, gate, rows, K, N, E, name, group=K).check()


# ---------------------------------------------------------------------------
# values that are not finite, on the large tiles
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("form,gate,rows,K,N,E,shape", [
    (4, 0, 5959, 384, 3824, 2, (4, 4, 4, 4)), (4, 1, 6274, 2048, 336, 8, (4, 4, 4, 4)),
    (8, 0, 5217, 384, 400, 13, (4, 2, 4, 4)), (8, 1, 5627, 128, 480, 13, (4, 2, 4, 4)),
    (8, 0, 5606, 2944, 1584, 2, (8, 4, 4, 4)), (8, 1, 7021, 3200, 608, 3, (8, 4, 4, 4))])
@pytest.mark.parametrize("name", ["float16", "bfloat16"])
def test_non_finite_rows_and_scales_stay_alone(form, gate, rows, K, N, E, shape, name):
    import torch
    say("non-finite", form, gate, rows, K, N, E, name)
    assert planned(w4.moe_gemm_describe(form, rows, K, N, E, gate, CUS))[:2] == (1, shape)
    c = Case(form, gate, rows, K, N, E, name)
    clean = c.run()
    live = int(c.starts[E])
    assert not clean[:live].isnan().any()
    source = np.arange(rows) if c.order is None else c.order // c.k
    if form == 8:
        c.a[3, K - 1], keep = 0x7F, (c.a[3, K - 1].item(), c.sa[70, K // 128 - 1].item())
        c.sa[70, K // 128 - 1] = float("nan")
    else:
        keep = c.a[3, K - 1].item(), c.a[70, 0].item()
        c.a[3, K - 1], c.a[70, 0] = float("nan"), float("inf")
    got = c.run()
    bad = torch.from_numpy(np.isin(source[:live], [3, 70])).cuda()
    nan = torch.from_numpy(source[:live] == 3).cuda()
    assert bad.any() and got[:live][nan].isnan().all()
    if form == 8:
        assert got[:live][bad].isnan().all()
    elif not gate:                       # gated, minus infinity times sigmoid(-infinity) = 0 is NaN
        assert not got[:live][bad].isfinite().any()
    assert torch.equal(got[:live][~bad], clean[:live][~bad])
    assert torch.equal(got[live:], clean[live:])
    if form == 8:
        c.a[3, K - 1], c.sa[70, K // 128 - 1] = keep
    else:
        c.a[3, K - 1], c.a[70, 0] = keep
    # one column's (8 bits: one block of columns') scale of the last expert
    e, col = E - 1, N - 1
    if form == 8:
        c.s[e, col // 128, 0] = float("nan")
        cols = np.flatnonzero(np.arange(2 * N if gate else N) // 128 == col // 128) % N
    else:
        c.s[e, -1, col] = float("nan")
        cols = np.array([col])
    got = c.run()[:live]
    bad = torch.zeros((live, N), dtype=torch.bool, device="cuda")
    bad[int(c.starts[e]):, torch.from_numpy(np.unique(cols)).cuda()] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], clean[:live][~bad])


@pytest.mark.parametrize("form,gate,rows,K,N,E,shape", [
    (4, 0, 5959, 384, 3824, 2, (4, 4, 4, 4)), (4, 1, 61, 640, 144, 5, (2, 2, 4, 4)),
    (8, 0, 5217, 384, 400, 13, (4, 2, 4, 4)), (8, 1, 7021, 3200, 608, 3, (8, 4, 4, 4))])
def test_tiles_with_index_tensors_of_anything(form, gate, rows, K, N, E, shape):
    """Starts out of order and orders of any whole numbers: nothing outside is
    written, and rows that are right get what they would."""
    import torch
    say("tiles nonsense", form, gate, rows, K, N, E)
    assert planned(w4.moe_gemm_describe(form, rows, K, N, E, gate, CUS))[:2] == (1, shape)
    c = Case(form, gate, rows, K, N, E, "float16")
    clean = c.run()
    rng = np.random.default_rng(0)
    starts = c.starts
    for i in range(4):
        c.starts = rng.integers(-2 ** 31, 2 ** 31, E + 1).astype(np.int32)
        if i % 2:
            c.starts = np.where(np.arange(E + 1) % 2 == 0, 0, rows + i).astype(np.int32)
        assert (c.run()[rows:] == 7.0).all(), i
    c.starts = starts
    if gate:                             # half the entries point anywhere: row 0 or some row
        bad = rng.random(rows) < 0.5
        c.order = np.where(bad, rng.integers(-2 ** 31, 2 ** 31, rows), c.order).astype(np.int32)
        got, ok = c.run(), torch.from_numpy(~bad).cuda()
        assert torch.equal(got[:rows][ok], clean[:rows][ok]) and (got[rows:] == 7.0).all()


# ---------------------------------------------------------------------------
# the gate far from zero
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("form,rows,K,shape", [
    (8, 3, 1024, (1, 2, 4, 4)), (8, 40, 1024, (2, 2, 4, 4)), (4, 3, 1024, (1, 2, 8, 3)),
    (4, 40, 1024, (1, 4, 4, 3)), (4, 40, 256, (2, 2, 4, 4))])
def test_gate_of_sums_far_from_zero(form, rows, K, shape):
    """Sums that FP32 holds exactly (one product of small numbers each), so that
    nothing but the gate and the output's rounding is off."""
    import torch
    N = 32
    say("gate", form, rows, K)
    assert planned(w4.moe_gemm_describe(form, rows, K, N, 1, 1, CUS))[1] == shape
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(rows, device="cuda") % 7 * 131 % K              # row p has 1 at channel at[p]
    p = torch.arange(rows, device="cuda")
    if form == 8:
        gate = torch.tensor([-80, -72, -60, -52, -40, -36, -30, -26, -20, -15, -10, -5, -2, -1, 0, 1,
                             2, 5, 10, 13, 20, 26, 32, 40, 48, 56, 64, 72, 80, 88, 96, 104.0])
        up = torch.tensor([1, -3, 7, 448.0]).repeat(8)
        codes = torch.cat([gate, up]).to(torch.float8_e4m3fn).view(torch.uint8)
        b = codes[:, None].repeat(1, K).cuda().contiguous()
        packed = w4.alloc_w8a8_packed(K, 2 * N)
        w4.w8a8_repack(b, packed)
        a = torch.zeros((rows, K), dtype=torch.uint8, device="cuda")
        a[p, at] = 0x38                                              # 1.0
        w4.w8a8_moe_gemm(a, torch.ones((rows, K // 128), device="cuda"), None, starts, packed,
                         torch.ones((1, 1, K // 128), device="cuda"), y, 1, w4.MOE_ACT_SILU_GATE)
        x = torch.cat([gate, up]).double()
    else:
        q = torch.arange(2 * N) % 16                                 # -8 .. 7
        words = torch.zeros((K // 8, 2 * N), dtype=torch.int64)
        for i in range(8):
            words |= q << (4 * i)
        words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32).cuda()
        packed = torch.empty(K * 2 * N // 8, dtype=torch.int32, device="cuda")
        w4.w4a16_repack(words, packed, K, 2 * N)
        s = torch.cat([torch.full((N,), 10.0), torch.full((N,), 3.0)]).to(torch.bfloat16)
        a = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
        a[p, at] = 1.0
        w4.w4a16_moe_gemm(a, None, starts, packed, s.repeat(K // 128, 1).cuda(), y, 1, 128,
                          w4.MOE_ACT_SILU_GATE)
        x = (q.double() - 8) * s.double()
    x = x.cuda()[None].repeat(rows, 1)
    want, d = _gated(x, torch.zeros_like(x), N)
    assert (want.abs() > 0).sum() > rows * N // 2
    _close(y, want, _rounding(want, d, "bfloat16"), "bfloat16", "gate")
