"""The reference of the 4-bit key/value cache, pinned to something other than
itself: hand-worked words, exact fractions, closed forms and invariants."""

from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest

from oracle import kv4_ref as ref


def test_quantise_a_hand_worked_row():
    # 16 evenly spaced values: scale 1, offset = -3 + 8, every code once
    x = np.arange(-3.0, 13.0, dtype=np.float32)
    q, p = ref.quantise(np.tile(x, 4))
    assert p.view(np.float16).tolist() == [1.0, 5.0]
    assert q.tolist() == list(range(16)) * 4


def test_quantise_constant_and_non_finite_rows():
    rows = np.zeros((5, 64), np.float32)
    rows[1] = 2.5
    rows[2, 7] = np.nan
    rows[3, 0] = np.inf
    rows[4] = 3e38 * np.where(np.arange(64) % 2, 1, -1)
    q, p = ref.quantise(rows)
    h = p.view(np.float16)
    assert (q[:4] == 8).all()
    assert h[0].tolist() == [0, 0] and h[1].tolist() == [0, 2.5]
    assert np.isnan(h[2:4].astype(float)).all()
    # far outside FP16: saturated, still finite
    assert np.isfinite(h[4].astype(float)).all() and set(q[4]) <= {0, 15}


def test_quantise_is_the_nearest_code():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 64)) * rng.uniform(0.01, 50, (200, 1))
         + rng.uniform(-9, 9, (200, 1))).astype(np.float32)
    q, p = ref.quantise(x)
    s, z = p.view(np.float16)[:, 0], p.view(np.float16)[:, 1]
    for r in range(0, 200, 7):
        fs, fz = Fraction(float(s[r])), Fraction(float(z[r]))
        for c in range(64):
            want = (Fraction(float(x[r, c])) - fz) / fs + 8
            got = int(q[r, c])
            # nearest, up to the two FP32 roundings of the quotient
            assert abs(want - got) <= Fraction(1, 2) + Fraction(1, 10 ** 5) \
                or got in (0, 15) and (want < 0) == (got == 0)


@pytest.mark.parametrize("D,page,heads", [(64, 16, 1), (128, 32, 3), (256, 64, 2)])
def test_layout_is_a_bijection(D, page, heads):
    """Every byte of the pages written belongs to exactly one token."""
    pages = 3
    touched = np.zeros(pages * heads * page * (D + 8), int)
    rng = np.random.default_rng(1)
    for slot in range(pages * page):
        a = rng.integers(0, 256, (pages, heads, page, D + 8)).astype(np.uint8)
        b = a.copy() ^ 0xFF
        x = rng.standard_normal((1, heads, D)).astype(np.float32)
        y = rng.standard_normal((1, heads, D)).astype(np.float32)
        before_a, before_b = a.copy(), b.copy()
        ref.store(a, [slot], x, y)
        ref.store(b, [slot], x, y)
        # a byte is written iff the two complementary backgrounds agree there
        same = (a == b).reshape(-1)
        touched += same
        assert same.sum() == heads * (D + 8)
        assert (a.reshape(-1)[~same] == before_a.reshape(-1)[~same]).all()
        assert (b.reshape(-1)[~same] == before_b.reshape(-1)[~same]).all()
        (kc, ks, kz), _ = ref.load(a, [slot])
        q, p = ref.quantise(x)
        assert (kc == q.astype(float) - 8).all()
        assert (ks == p.view(np.float16)[..., 0].astype(float)).all()
        assert (kz == p.view(np.float16)[..., 1].astype(float)).all()
    assert (touched == 1).all()


def test_layout_hand_worked_addresses():
    """Token 21 of page 1 (unit 1, row 5), head 1 of 2, D = 64."""
    cache = np.zeros((2, 2, 32, 72), np.uint8)
    x = np.zeros((1, 2, 64), np.float32)
    x[0, 1] = np.tile(np.arange(16.0), 4)           # codes 0..15 four times
    ref.store(cache, [32 + 21], x, x)
    flat = cache.reshape(-1)
    unit = ((1 * 2 + 1) * 2 + 1) * 1152
    word = [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert flat[unit + 5 * 32: unit + 5 * 32 + 8].tolist() == word
    # values: group 1 (tokens 4..7), word w, token 1 of the group
    base = unit + 512
    for w in range(8):
        at = base + ((1 * 8 + w) * 4 + 1) * 4
        assert flat[at: at + 4].tolist() == word[4 * (w % 2): 4 * (w % 2) + 4]
    for off in (1024, 1088):
        assert flat[unit + off + 20: unit + off + 24].view(np.float16).tolist() == [1.0, 8.0]


@pytest.mark.parametrize("pairs", [0, 1])
def test_rope_is_a_rotation_of_complex_numbers(pairs):
    rng = np.random.default_rng(2)
    T, H, D, sections = 5, 2, 64, (4, 6, 6)
    x = rng.standard_normal((T, H, D))
    pos = rng.integers(0, 1000, (3, T))
    freq = 10000.0 ** (-np.arange(16) / 16)
    y = ref.rope(x, pos, freq, sections, pairs)
    assert (y[..., 32:] == x[..., 32:]).all()
    for i in range(16):
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + 16)
        axis = 0 if i < 4 else 1 if i < 10 else 2
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[axis] * freq[i])[:, None]
        assert np.allclose(y[..., a] + 1j * y[..., b], z, atol=1e-12)
    back = ref.rope(y, -pos, freq, sections, pairs)
    assert np.allclose(back, x, atol=1e-12)


def _cache(rng, pages, heads, page, D):
    cache = rng.integers(0, 256, (pages, heads, page, D + 8)).astype(np.uint8)
    n = pages * page
    ref.store(cache, list(range(n)), rng.standard_normal((n, heads, D)).astype(np.float32),
              rng.standard_normal((n, heads, D)).astype(np.float32))
    return cache


def test_attention_against_explicit_sums():
    rng = np.random.default_rng(3)
    cache = _cache(rng, 4, 2, 16, 64)
    table = np.array([[2, 0, 1], [3, -1, -1]], np.int32)
    lens, starts = [37, 5], [0, 3, 4]
    q = rng.standard_normal((4, 4, 64))
    o, lse, *_ = ref.attention(q, cache, table, lens, starts, 0.125, window=20)
    for t, (b, pos) in enumerate([(0, 34), (0, 35), (0, 36), (1, 4)]):
        for h in range(4):
            den, num = 0.0, np.zeros(64)
            for j in range(max(0, pos - 19), pos + 1):
                slot = int(table[b, j // 16]) * 16 + j % 16
                part_k, part_v = ref.load(cache, [slot])
                k, v = ref.values_of(part_k)[0, h // 2], ref.values_of(part_v)[0, h // 2]
                w = np.exp(0.125 * float(q[t, h] @ k))
                den += w
                num += w * v
            assert np.allclose(o[t, h], num / den, atol=1e-12)
            assert np.isclose(lse[t, h], np.log(den), atol=1e-12)


def test_attention_of_nothing_and_of_one_key():
    rng = np.random.default_rng(4)
    cache = _cache(rng, 2, 1, 16, 64)
    table = np.array([[1], [0], [-1]], np.int32)
    q = rng.standard_normal((4, 1, 64))
    # request 0 has two queries for one token: the first sees nothing
    o, lse, *_ = ref.attention(q, cache, table, [1, 0, 4], [0, 2, 3, 4], 1.0)
    _, v = ref.load(cache, [16])
    assert (o[0] == 0).all() and lse[0, 0] == -np.inf
    assert np.allclose(o[1, 0], ref.values_of(v)[0, 0])
    assert (o[2:] == 0).all() and (lse[2:] == -np.inf).all()


def test_tables_conserve_pages():
    rng = np.random.default_rng(5)
    page, width, pages, B = 16, 6, 40, 9
    table = np.full((B, width), -1, np.int32)
    ring, state = np.arange(pages, dtype=np.int32), np.array([7, pages, 0, 0], np.int32)
    ring = np.roll(ring, 7)
    lens = np.zeros(B, np.int32)
    for _ in range(200):
        want = np.clip(lens + rng.integers(-40, 30, B), 0, 110).astype(np.int32)
        new, table, ring, state, qs, slots, pos = ref.tables(lens, want, table, ring, state, 400,
                                                             page)
        held = [int(p) for b in range(B) for p in table[b, : -(-int(new[b]) // page)]]
        free = [int(ring[(state[0] + i) % pages]) for i in range(state[1])]
        assert sorted(held + free) == list(range(pages))
        assert state[2] == (new != want).sum()
        for b in range(B):
            for i in range(qs[b + 1] - qs[b]):
                p = int(lens[b]) + i
                assert pos[qs[b] + i] == p
                s = slots[qs[b] + i]
                assert s == (table[b, p // page] * page + p % page if new[b] == want[b] else -1)
        assert (slots[qs[B]:] == -1).all()
        lens = new
