"""Scheduler steps with more new tokens than the token buffers hold: the
reference's rule, worked by hand."""

from __future__ import annotations

import numpy as np

from oracle import kv4_ref as ref


def _step(lens, want, capacity, page=16, width=4, pages=12, count=None):
    used = [-(-max(0, n) // page) for n in lens]
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = np.arange(at, at + n)
        at += n
    ring = np.concatenate((np.arange(at, pages), np.full(at, -9))).astype(np.int32)
    state = [0, pages - at if count is None else count, 0, 0]
    return table, ring, ref.tables(lens, want, table, ring, state, capacity, page)


def test_a_request_whose_tokens_do_not_all_fit_is_refused():
    table, ring, out = _step([0, 0, 5], [32, 32, 6], 40)
    lens, t, r, state, q_start, slots, pos = out
    # the first takes pages 1 and 2; the second's last 24 tokens have no room
    assert lens.tolist() == [32, 0, 5]
    assert t[0].tolist() == [1, 2, -1, -1] and (t[1:] == table[1:]).all() and (r == ring).all()
    assert state.tolist() == [2, 9, 2, 0]
    assert q_start.tolist() == [0, 32, 40, 40]
    assert slots.tolist() == list(range(16, 48)) + [-1] * 8
    assert pos.tolist() == list(range(32)) + list(range(8))


def test_a_step_that_fits_exactly_refuses_nothing():
    _, _, out = _step([0, 0, 5], [32, 7, 6], 40)
    lens, _, _, state, q_start, slots, _ = out
    assert lens.tolist() == [32, 7, 6] and state[2] == 0 and q_start.tolist() == [0, 32, 39, 40]
    assert (slots >= 0).all()


def test_requests_that_do_not_grow_are_served_whatever_the_capacity():
    # the first fills more than there is; the second stays, the third shrinks, the last grows
    _, _, out = _step([1, 40, 40, 16], [60, 40, 3, 17], 16)
    lens, _, ring, state, q_start, slots, _ = out
    assert lens.tolist() == [1, 40, 3, 16]
    assert state.tolist() == [0, 4 + 2, 2, 0]
    assert ring[4:6].tolist() == [5, 6]                  # the third's pages 1 and 2
    assert q_start.tolist() == [0, 16, 16, 16, 16] and (slots == -1).all()


def test_a_request_refused_for_want_of_pages_still_takes_its_rows():
    # its rows count in q_start, so the one after it does not fit either
    _, _, out = _step([0, 0, 0], [16, 16, 4], 34, count=1)
    lens, _, _, state, q_start, slots, _ = out
    assert lens.tolist() == [16, 0, 0] and state.tolist() == [1, 0, 2, 0]
    assert q_start.tolist() == [0, 16, 32, 34] and slots.tolist() == list(range(16)) + [-1] * 18


def test_no_room_at_all():
    _, _, out = _step([0, 8, 8], [1, 8, 0], 0)
    assert out[0].tolist() == [0, 8, 0] and out[3].tolist() == [0, 11, 1, 0]
    assert out[4].tolist() == [0, 0, 0, 0]


def test_no_slot_is_left_unwritten_below_a_length():
    """Whatever the capacity, every token below lens_out was below lens or has
    its slot in this step."""
    rng = np.random.default_rng(0)
    for _ in range(200):
        B = int(rng.integers(1, 7))
        lens = rng.integers(0, 50, B)
        want = np.clip(lens + rng.integers(-20, 30, B), 0, 80)
        _, _, out = _step(lens, want, int(rng.integers(0, 60)), pages=64)
        new, table, _, _, q_start, slots, pos = out
        for b in range(B):
            given = {int(pos[t]): int(slots[t]) for t in range(q_start[b], q_start[b + 1])}
            for p in range(int(lens[b]), int(new[b])):
                assert given[p] == table[b, p // 16] * 16 + p % 16
            if new[b] < want[b]:
                assert new[b] == lens[b] and all(s == -1 for s in given.values())
