"""Which calls are refused because their tensors share memory: those that do,
and no others where the strides are alike, as in parts of one buffer."""

from __future__ import annotations

import random

import pytest

import weight_only_int4_gemm_amd as w4
from tests.test_kv4_abi import A, ATTEND, DEVICE, FUSED, ROPE, SHAPE, _sections


@pytest.fixture(scope="module", autouse=True)
def no_device():
    """Fake addresses: accepted calls must end at the first look at a device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("without a device only")


def _elements(at, token, head, T, H, D):
    return {at + t * token + h * head + c for t in range(T) for h in range(H) for c in range(D)}


def test_rope_append_in_place_in_a_buffer_interleaved_by_head():
    """[T][heads][q, k, v][D], the layout of projections fused head by head."""
    call = w4.load().kv4_rope_append
    for T, H, D in ((10, 8, 128), (1, 8, 128), (7, 1, 64), (4096, 32, 128)):
        row = dict(q_token=3 * H * D, k_token=3 * H * D, v_token=3 * H * D, qo_token=3 * H * D,
                   q_head=3 * D, k_head=3 * D, v_head=3 * D, qo_head=3 * D)
        args = {**FUSED, **row, "T": T, "Hq": H, "H": H, "D": D, "Q": A[0], "K": A[0] + 2 * D,
                "V": A[0] + 4 * D, "Qout": A[0], "sections": _sections(D // 2)}
        assert call(*args.values()) == DEVICE, (T, H, D)
        # the same strides over the keys, the values, or between two parts
        for over in (2 * D, 4 * D, D, 16):
            assert call(*{**args, "Qout": A[0] + over}.values()) == SHAPE, (T, H, D, over)


def test_attention_into_another_part_of_the_queries_buffer():
    call = w4.load().kv4_attention
    T, H, D = 6, 8, 128
    for head, token, step in ((D, 3 * H * D, H * D), (3 * D, 3 * H * D, D)):
        args = {**ATTEND, "q_token": token, "q_head": head, "o_token": token, "o_head": head,
                "T": T, "Hq": H, "Q": A[0], "O": A[0] + 4 * step}
        assert call(*args.values()) == DEVICE
        for over in (0, 16, 2 * step - 16, 2 * token):
            assert call(*{**args, "O": A[0] + over}.values()) == SHAPE, over


@pytest.mark.parametrize("seed", range(4))
def test_rotation_is_refused_where_elements_are_shared(seed):
    """Random layouts against sets of elements."""
    rng, call = random.Random(seed), w4.load().kv4_rope
    accepted = refused = 0
    for _ in range(1500):
        T, H, D = rng.randint(1, 4), rng.randint(1, 4), 64
        kind = rng.randrange(4)
        pad = rng.choice((0, 8, 64, 72, 128, 200))
        if kind < 2:                                    # heads inside tokens
            head = D + pad
            token = H * head + rng.choice((0, 8, 64, 128, 600))
        else:                                           # tokens inside heads
            token = D + pad
            head = T * token + rng.choice((0, 8, 64, 128, 600))
        other = (token, head)
        if kind % 2 and rng.random() < 0.5:
            other = (token + 64 * H, head + 64 * T)
        by = 8 * rng.randint(-90, 90) if rng.random() < 0.7 else 64 * rng.randint(-9, 9)
        base = 1 << 20
        x = _elements(base, token, head, T, H, D)
        y = _elements(base + by, *other, T, H, D)
        args = {**ROPE, "X": A[0] + 2 * base, "x_token": token, "x_head": head,
                "Y": A[0] + 2 * (base + by), "y_token": other[0], "y_head": other[1], "T": T,
                "H": H, "D": D, "sections": _sections(32), "axes": 1}
        rc = call(*args.values())
        shared = bool(x & y) and not (by == 0 and other == (token, head))
        if shared:
            assert rc == SHAPE, args
        elif other == (token, head):
            assert rc == DEVICE, args
        accepted += rc == DEVICE
        refused += rc == SHAPE
    assert accepted > 200 and refused > 200


def test_outputs_over_the_small_inputs():
    """Positions, frequencies and slots are read while rows are written."""
    lib = w4.load()
    for name, out in (("positions", "Y"), ("inv_freq", "Y")):
        assert lib.kv4_rope(*{**ROPE, name: ROPE[out] + 64}.values()) == SHAPE, name
    for name in ("positions", "inv_freq", "slots"):
        for out in ("Qout", "cache"):
            assert lib.kv4_rope_append(*{**FUSED, name: FUSED[out] + 64}.values()) == SHAPE, name
    assert lib.kv4_rope(*ROPE.values()) == DEVICE
    assert lib.kv4_rope_append(*FUSED.values()) == DEVICE
