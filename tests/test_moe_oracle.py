"""The reference of the expert layers and 8-bit products, pinned to something
other than itself: hand-worked values, torch's own e4m3 conversion, invariants."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import moe_ref as ref


def test_e4m3_against_torch():
    import torch
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = ref.e4m3_value(codes)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got).sum() == 2
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    # every midpoint, and next to it on both sides
    v = ref.e4m3_value(np.arange(0x7F))
    mid = ((v[1:] + v[:-1]) / 2).astype(np.float32)
    x = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(999)),
                        v.astype(np.float32)])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_code(x), want)


def test_quantise_hand_worked():
    x = np.zeros((4, 256), np.float32)
    x[0, 0], x[0, 1], x[0, 130] = 448.0, 1.0, -896.0
    x[2, 5] = np.inf
    x[3, 255] = np.nan
    q, s = ref.quantise(x)
    assert s[0].tolist() == [1.0, 2.0]
    assert q[0, 0] == 0x7E and q[0, 1] == 0x38 and q[0, 130] == 0xFE
    assert s[1].tolist() == [2.0 ** -126] * 2 and not q[1].any()
    assert np.isnan(s[2, 0]) and s[2, 1] == np.float32(2.0 ** -126) and not q[2].any()
    assert s[3, 0] == np.float32(2.0 ** -126) and np.isnan(s[3, 1])


def test_quantise_is_within_half_a_step():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 256)) * np.exp(rng.uniform(-20, 20, (50, 1)))).astype(np.float32)
    q, s = ref.quantise(x)
    y = ref.dequantise(q, s)
    steps = np.repeat(s.astype(float), 128, 1)
    # half a step of 2^-4 relative, or half the smallest step
    assert (np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * steps) * 1.0001).all()


@pytest.mark.parametrize("N,K", [(16, 128), (48, 384)])
def test_repack_is_a_bijection_in_the_order_of_the_instruction(N, K):
    rng = np.random.default_rng(1)
    q = rng.integers(0, 256, (N, K)).astype(np.uint8)
    p = ref.repack8(q)
    # lane l of half h of block (n16, kb): 16 consecutive in-features of one column
    for n16, kb, h, lane in ((0, 0, 0, 0), (N // 16 - 1, K // 128 - 1, 1, 63), (0, K // 128 - 1, 1, 17)):
        at = ((n16 * (K // 128) + kb) * 2 + h) * 1024 + lane * 16
        k0 = kb * 128 + h * 64 + lane // 16 * 16
        assert np.array_equal(p[at:at + 16], q[n16 * 16 + lane % 16, k0:k0 + 16])
    assert np.array_equal(np.sort(p), np.sort(q.reshape(-1)))


def test_route_hand_worked():
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = ref.route(x, None, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w = ref.route(x, None, 3, renorm=False, scale=2.0)
    assert ids.tolist() == [[2, 1, 0]] and np.allclose(w, [[1.0, 0.5, 0.25]])
    # a bias chooses, the score weighs
    ids, w = ref.route(x, np.array([0, 0, 0, 9.0]), 1, renorm=False)
    assert ids.tolist() == [[3]] and np.allclose(w, [[0.125]])
    ids, w = ref.route(np.array([[0.0, np.log(3.0)]]), None, 1, softmax=False, renorm=False)
    assert ids.tolist() == [[1]] and np.allclose(w, [[0.75]])


def test_route_masked_and_tied():
    inf, nan = np.inf, np.nan
    ids, w = ref.route(np.array([[-inf, nan, 3.0, -inf]]), None, 3)
    assert ids.tolist() == [[2, -1, -1]] and w.tolist() == [[1, 0, 0]]
    ids, w = ref.route(np.full((1, 4), -inf), None, 2)
    assert ids.tolist() == [[-1, -1]] and not w.any()
    ids, w = ref.route(np.zeros((1, 6)), None, 3)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 1 / 3)
    ids, w = ref.route(np.array([[0, inf, 1, inf]]), None, 3, renorm=False)
    assert ids.tolist() == [[1, 3, 2]] and w.tolist() == [[0.5, 0.5, 0]]


def test_route_groups():
    # groups of two: marks by best one 3, 4, 1; by the two best 6, 4.5, 2
    x = np.array([[3, 3, 4, .5, 1, 1]]) / 10
    b = np.zeros(6)
    kind = dict(softmax=False, groups=3, top_groups=1, renorm=False)
    assert ref.route(x, b, 2, group_best=1, **kind)[0].tolist() == [[2, 3]]
    assert ref.route(x, b, 2, group_best=2, **kind)[0].tolist() == [[0, 1]]
    assert ref.route(x, b, 3, group_best=2, **kind)[0].tolist() == [[0, 1, -1]]


def test_tables_are_a_stable_sort():
    rng = np.random.default_rng(2)
    ids = rng.integers(-1, 9, (40, 3))
    starts, order, where = ref.tables(ids, 8)
    flat = ids.reshape(-1)
    kept = order[:starts[8]]
    assert (order[starts[8]:] == -1).all()
    assert np.array_equal(kept, [i for i in np.argsort(np.where((flat < 0) | (flat > 7), 99, flat),
                                                      kind="stable")][:starts[8]])
    for i, p in enumerate(where.reshape(-1)):
        assert (p == -1 and not 0 <= flat[i] < 8) or order[p] == i


def test_expert_rows_and_combine():
    rng = np.random.default_rng(3)
    A, W = rng.standard_normal((5, 8)), rng.standard_normal((3, 8, 4))
    ids = np.array([[0, 2], [2, -1], [0, 1], [1, 0], [2, 1]])
    starts, order, where = ref.tables(ids, 3)
    y, _ = ref.expert_rows(A, order, starts, W, 2, 10)
    w = rng.uniform(size=(5, 2))
    got = ref.combine(y, where, w)
    for t in range(5):
        want = sum(w[t, j] * (A[t] @ W[ids[t, j]]) for j in range(2) if ids[t, j] >= 0)
        assert np.allclose(got[t], want)
