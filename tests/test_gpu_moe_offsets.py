"""Expert layers and 8-bit products where offsets pass 32 bits: weights of many
experts, rows gathered from and stored far behind the start of their tensors.
Only what lies there is looked at.  Tolerances as in test_gpu_moe_tiles.py."""

from __future__ import annotations

import gc

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import moe_ref as ref
from tests import test_gpu_moe_tiles as tiles
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

PAST = 1 << 32


@pytest.fixture(autouse=True)
def _free():
    import torch
    yield
    gc.collect()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("form,name", [(8, "bfloat16"), (4, "float16"), (4, "bfloat16")])
@pytest.mark.parametrize("gate", [0, 1])
def test_experts_far_apart(form, name, gate):
    import torch
    K, W = 4096, 8192
    N = W // 2 if gate else W
    E = 130 if form == 8 else 260
    rows, a_rows = (1 << 20) // (1 if gate else 2) + 77, (1 << 20) + 64
    say("experts offsets", form, name, gate, w4.moe_gemm_describe(form, rows, K, N, E, gate))
    g = tiles._gen(form + gate)
    used = {5: (rows - 43, rows - 40), E - 1: (rows - 40, rows - 3)}
    starts = np.full(E + 1, rows - 43, np.int32)
    starts[6:], starts[E] = rows - 40, rows - 3
    order = np.zeros(rows, np.int32)
    order[rows - 43:] = a_rows - 1 - np.arange(43) * 3
    dt = getattr(torch, name)
    y = torch.full((rows + 1, N), 7.0, dtype=dt, device="cuda")
    assert y.numel() >= PAST
    idx = torch.from_numpy(order).cuda(), torch.from_numpy(starts).cuda()
    live = torch.from_numpy(order[rows - 43:rows - 3]).cuda().long()
    act = w4.MOE_ACT_SILU_GATE if gate else w4.MOE_ACT_NONE
    weights = {}
    if form == 8:
        a = torch.zeros((a_rows, K), dtype=torch.uint8, device="cuda")
        sa = torch.zeros((a_rows, K // 128), device="cuda")
        a[live], sa[live] = tiles._codes((40, K), g), tiles._scales((40, K // 128), g)
        packed = torch.empty((E, K * W), dtype=torch.uint8, device="cuda")
        s = torch.zeros((E, W // 128, K // 128), device="cuda")
        for e in used:
            b, s[e] = tiles._codes((W, K), g), tiles._scales((W // 128, K // 128), g)
            w4.w8a8_repack(b, packed[e])
            weights[e] = tiles._weights8(b, s[e]), None
        x = tiles._rows8(a[live], sa[live])
        w4.w8a8_moe_gemm(a, sa, *idx, packed, s, y[:rows], 1, act)
    else:
        a = torch.zeros((a_rows, K), dtype=dt, device="cuda")
        a[live] = tiles._randn((40, K), g).to(dt)
        packed = torch.empty((E, K * W // 8), dtype=torch.int32, device="cuda")
        s = torch.zeros((E, K // 128, W), dtype=dt, device="cuda")
        for e in used:
            b = torch.randint(-2 ** 31, 2 ** 31, (K // 8, W), device="cuda", generator=g,
                              dtype=torch.int64).to(torch.int32)
            s[e] = (torch.rand((K // 128, W), device="cuda", generator=g) * 0.015 + 0.005).to(dt)
            w4.w4a16_repack(b, packed[e], K, W)
            weights[e] = tiles._int4(b, s[e], 128)
        x = a[live].double()
        w4.w4a16_moe_gemm(a, *idx, packed, s, y[:rows], 1, 128, act)
    assert a.numel() * a.element_size() >= PAST and packed.numel() * packed.element_size() >= PAST
    for e, (lo, hi) in used.items():
        r, (w, steps) = x[lo - rows + 43:hi - rows + 43], weights[e]
        want = r @ w
        d = tiles._sums(K) * (r.abs() @ w.abs())
        if form == 4 and name == "bfloat16":
            d = d + 320 * 2 * tiles.U * 279 * (r.abs() @ steps)
        if gate:
            want, d = tiles._gated(want, d, N)
        tiles._close(y[lo:hi], want, tiles._rounding(want, d, name), name, e)
    assert (y[rows - 3:] == 7.0).all()
    for lo in range(0, rows - 43, 1 << 16):                  # nothing else is written
        assert (y[lo:min(lo + (1 << 16), rows - 43)] == 7.0).all(), lo


def test_dense_rows_far_apart():
    import torch
    M, K, N = (1 << 19) + 13, 128, 8192
    say("dense offsets", w4.w8a8_describe(M, K, N))
    g = tiles._gen(1)
    a, sa = tiles._codes((M, K), g), tiles._scales((M, 1), g)
    b, sb = tiles._codes((N, K), g), tiles._scales((N // 128, 1), g)
    packed = w4.alloc_w8a8_packed(K, N)
    w4.w8a8_repack(b, packed)
    c = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    assert c.numel() > PAST
    w4.w8a8_gemm(a, sa, packed, sb, c[:M], w4.alloc_w8a8_workspace(M, K, N))
    w = tiles._weights8(b, sb)
    for at in (slice(0, 200), slice((1 << 18) - 100, (1 << 18) + 100), slice(M - 200, M)):
        x = tiles._rows8(a[at], sa[at])
        want = x @ w
        d = tiles._sums(K) * (x.abs() @ w.abs())
        tiles._close(c[at], want, tiles._rounding(want, d, "bfloat16"), "bfloat16", at)
    assert (c[M:] == 7.0).all()


def test_repack_of_more_than_32_bits():
    import torch
    N, K = (1 << 18) + 48, 16384
    say("repack offsets", N, K)
    b = torch.zeros((N, K), dtype=torch.uint8, device="cuda")
    q = np.random.default_rng(0).integers(0, 256, (48, K)).astype(np.uint8)
    b[N - 48:] = torch.from_numpy(q).cuda()
    out = torch.full((N * K + 16,), 0x55, dtype=torch.uint8, device="cuda")
    assert N * K > PAST
    w4.w8a8_repack(b, out[:N * K])
    tail = out[(N - 48) * K:].cpu().numpy()
    assert np.array_equal(tail[:-16], ref.repack8(q)) and (tail[-16:] == 0x55).all()
    assert not out[(N - 64) * K:(N - 48) * K].any()


def test_quantize_rows_far_apart():
    import torch
    T, K = (1 << 18) + 5, 16384
    say("quantize offsets", T, K)
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    x[T - 8:] = torch.from_numpy(rng.standard_normal((8, K)).astype(np.float32)).cuda()
    q = torch.full((T, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((T, K // 128), -1.0, device="cuda")
    assert T * K > PAST
    w4.w8a8_quantize(x, q, s)
    want_q, want_s = ref.quantise(x[T - 8:].float().cpu().numpy())
    assert np.array_equal(q[T - 8:].cpu().numpy(), want_q)
    assert np.array_equal(s[T - 8:].cpu().numpy(), want_s)
    assert not q[:T - 8].any() and (s[:T - 8] == 2.0 ** -126).all()


def test_combine_rows_far_apart():
    import torch
    N, far = 8192, (1 << 19) + 77
    g = tiles._gen(3)
    say("combine offsets", far, N)
    y = torch.zeros((far, N), dtype=torch.bfloat16, device="cuda")
    assert y.numel() > PAST
    y[far - 4:] = tiles._randn((4, N), g).to(torch.bfloat16)
    where = torch.tensor([[far - 1, far - 3], [far - 4, far], [0, far - 2]], dtype=torch.int32,
                         device="cuda")
    weights = torch.tensor([[0.25, 0.5], [0.75, 2.0], [1.0, 0.3]], device="cuda")
    out = torch.empty((3, N), dtype=torch.bfloat16, device="cuda")
    w4.moe_combine(y, where, weights, out)
    w = weights.double() * (where < far)
    rows = y[where.clamp(max=far - 1).long()].double()
    want = (rows * w[..., None]).sum(1)
    S = (rows.abs() * w[..., None]).sum(1)
    h = 2.0 ** -8
    tiles._close(out, want, 6 * tiles.U * S + h * want.abs() + 2.0 ** -134, "bfloat16", "combine")
    # and tokens far apart
    del y, out
    y = tiles._randn((7, N), g).to(torch.bfloat16)
    where = torch.full((far, 1), -1, dtype=torch.int32, device="cuda")
    where[far - 3:] = torch.tensor([[6], [0], [3]], dtype=torch.int32, device="cuda")
    out = torch.full((far + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    w4.moe_combine(y, where, torch.ones((far, 1), device="cuda"), out[:far])
    assert torch.equal(out[far - 3:far], y[[6, 0, 3]]) and (out[far:] == 7.0).all()
    for lo in range(0, far - 3, 1 << 16):
        assert not out[lo:min(lo + (1 << 16), far - 3)].any(), lo


@pytest.mark.parametrize("name", ["bfloat16", "float32"])
def test_route_rows_far_apart(name):
    import torch
    T, E, k, row = 19, 96, 4, (1 << 28) + 1
    say("route offsets", name)
    room = torch.empty(((T - 1) * row + E,), dtype=getattr(torch, name), device="cuda")
    x = room.as_strided((T, E), (row, 1))
    assert room.numel() > PAST
    x.copy_(tiles._randn((T, E), tiles._gen(4)))
    near = x.contiguous()
    got = []
    for logits in (x, near):
        ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        weights = torch.zeros((T, k), device="cuda")
        w4.moe_route(logits, None, ids, weights)
        got.append((ids, weights))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert (got[0][0].sort(-1).values.diff(dim=-1) > 0).all()


def test_tables_of_the_most_choices():
    import torch
    T, k, E = 1 << 21, 8, 1024
    say("tables most", T * k, E)
    rng = np.random.default_rng(1)
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)
    starts, order, where = w4.alloc_moe_tables(T, k, E)
    w4.moe_tables(torch.from_numpy(ids).cuda(), starts, order, where)
    flat = np.where((ids < 0) | (ids >= E), E, ids).reshape(-1)
    o = np.argsort(flat, kind="stable").astype(np.int32)
    n = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])])
    wh = np.full(flat.size, -1, np.int32)
    wh[o[:n[E]]] = np.arange(n[E])
    o[n[E]:] = -1
    assert np.array_equal(starts.cpu().numpy(), n)
    assert np.array_equal(order.cpu().numpy(), o)
    assert np.array_equal(where.cpu().numpy().reshape(-1), wh)
