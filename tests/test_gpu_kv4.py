"""The 4-bit key/value cache operators on the GPU against the reference in
64 bits (stored forms and whole numbers bit for bit).

Tolerances, derived from the arithmetic:
* rotation: cos and sin rounded to FP32, two products and a sum in FP32, one
  rounding of the result: eps/2 |y| + 4 2^-24 (|x1| + |x2|);
* attention: the output's rounding eps/2 |o|; the rounding of each weight to
  FP16, 2^-11 of sum p s |c - 8| (BF16 calls; FP16 calls carry the rounding's
  remainder too: 2^-21), at least half FP16's smallest step, 2^-25 of the
  largest weight for each of n keys; scores summed in FP32, where eight roundings of the
  largest magnitude in them move every p by that much; and sums of n terms in
  FP32, taken as 64 + n/32 roundings of the sum of magnitudes;
* lse: the same score error and 64 roundings of 1 + |lse|.
"""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import kv4_ref as ref
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
    return t, t.float().cpu().numpy()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def half_eps(name):
    return float(_torch().finfo(_dtype(name)).eps) / 2


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

def _run_tables(lens, want, table, ring, state, capacity, page, alias):
    torch = _torch()
    i32 = torch.int32
    d = [cuda(np.asarray(x, np.int32)) for x in (lens, want, table, ring, state)]
    B = table.shape[0]
    if B == 0:
        d[2] = torch.empty(table.shape, dtype=i32, device="cuda")
    lens_out = d[0] if alias else torch.full((B,), -7, dtype=i32, device="cuda")
    state_out = d[4] if alias else torch.zeros(4, dtype=i32, device="cuda")
    q_start = torch.full((B + 1,), -7, dtype=i32, device="cuda")
    slots = torch.full((capacity,), -7, dtype=i32, device="cuda")
    pos = torch.full((capacity,), -7, dtype=i32, device="cuda")
    w4.kv4_tables(d[0], d[1], d[2], d[3], d[4], lens_out, state_out, q_start, slots, pos, page)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (lens_out, d[2], d[3], state_out, q_start, slots, pos)]


TABLE_NAMES = ("lens_out", "table", "ring", "state_out", "q_start", "slots", "positions")


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,page,width,grow,pages", [
    (1, 16, 1, 1, 1), (3, 16, 4, 9, 64), (64, 64, 33, 1, 64 * 33), (255, 32, 9, 70, 1200),
    (256, 1024, 3, 2000, 500), (257, 16, 65, 200, 9000), (1000, 16, 40, 100, 20000),
    (4096, 128, 5, 3, 20000)])
def test_tables_match_the_reference(B, page, width, grow, pages, alias):
    rng = np.random.default_rng(B + page)
    lens = rng.integers(0, width * page + 1, B)
    kind = rng.random(B)
    want = np.where(kind < 0.6, lens + rng.integers(0, grow + 1, B),
                    np.where(kind < 0.8, np.maximum(0, lens - rng.integers(0, 3 * page, B)), 0))
    used = -(-lens // page)
    while used.sum() > pages:                       # give up the last requests' pages
        b = int(np.flatnonzero(used)[-1])
        lens[b] = want[b] = used[b] = 0
    ids = rng.permutation(pages)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, : used[b]] = ids[at: at + used[b]]
        at += used[b]
    free = ids[at:]
    head = int(rng.integers(0, pages))
    ring = np.full(pages, -9, np.int32)
    ring[(head + np.arange(len(free))) % pages] = free
    total = int(np.maximum(0, want - lens).sum())
    for capacity in (max(0, total - 5), total + 70):
        say("tables", B, page, width, capacity, alias)
        state = [head, len(free), 0, 0]
        got = _run_tables(lens, want, table, ring, state, capacity, page, alias)
        expect = ref.tables(lens, want, table, ring, state, capacity, page)
        for name, g, e in zip(TABLE_NAMES, got, expect):
            assert np.array_equal(g, e), name


def test_tables_out_of_pages_and_out_of_range():
    page, width, pages = 16, 4, 10
    table = np.array([[0, -1, -1, -1], [1, 2, -1, -1], [3, 999, -1, -1], [-5, -1, -1, -1],
                      [-1, -1, -1, -1], [4, 5, -1, -1]], np.int32)
    ring = np.array([6, 7, 8, 9, 0, 0, 0, 0, 0, 0], np.int32)
    lens = [16, 20, 17, 3, -4, 30]
    want = [48, 200, 18, 4, 2147483647, 31]       # two pages; too long; bad ids; too long; none
    for state in ([0, 4, 0, 0], [0, 1, 0, 0], [0, 0, 0, 0], [7, 3, 0, 0]):
        got = _run_tables(lens, want, table, ring, state, 300, page, False)
        expect = ref.tables(lens, want, table, ring, state, 300, page)
        for name, g, e in zip(TABLE_NAMES, got, expect):
            assert np.array_equal(g, e), (name, state)
    got = _run_tables([], [], np.zeros((0, 4), np.int32), ring, [2, 3, 0, 0], 5, page, False)
    assert got[3].tolist() == [2, 3, 0, 0] and got[4].tolist() == [0]
    assert got[5].tolist() == [-1] * 5 and got[6].tolist() == [0] * 5


def test_tables_a_life_in_place_under_a_graph():
    """Steps replayed from one graph with in-place state equal the reference's."""
    torch = _torch()
    rng = np.random.default_rng(6)
    B, page, width, pages, capacity = 37, 16, 12, 260, 4096
    table, ring, state = w4.alloc_kv4_pages(pages, B, width)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, want = torch.zeros(B, **i32), torch.zeros(B, **i32)
    q_start, slots, pos = (torch.zeros(n, **i32) for n in (B + 1, capacity, capacity))
    r_lens, r_table, r_ring, r_state = (x.cpu().numpy() for x in (lens, table, ring, state))

    def step():
        w4.kv4_tables(lens, want, table, ring, state, lens, state, q_start, slots, pos, page)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(25):
        w = np.clip(r_lens + rng.integers(-60, 70, B), 0, 200).astype(np.int32)
        want.copy_(torch.from_numpy(w))
        graph.replay()
        torch.cuda.synchronize()
        expect = ref.tables(r_lens, w, r_table, r_ring, r_state, capacity, page)
        for name, g, e in zip(TABLE_NAMES, (lens, table, ring, state, q_start, slots, pos), expect):
            assert np.array_equal(g.cpu().numpy(), e), (i, name)
        r_lens, r_table, r_ring, r_state = expect[:4]


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------

def _rope_inputs(rng, T, axes, half, far):
    cut = sorted(int(c) for c in rng.integers(0, half + 1, axes - 1))
    sections = tuple(np.diff([0, *cut, half]).tolist())
    pos = rng.integers(-5, far, (axes, T)).astype(np.int32)
    freq = 10000.0 ** (-np.arange(half) / half)
    return sections, pos, freq


def _rope_bound(y, x, half, pairs, name):
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    size = np.zeros_like(y)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return half_eps(name) * np.abs(y) + 4 * U * size + 2.0 ** -25


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,H,D,rot,axes,pairs,far", [
    (1, 1, 64, 64, 1, 0, 100), (5, 3, 64, 32, 2, 1, 5000), (67, 8, 128, 128, 3, 0, 1000000),
    (67, 8, 128, 128, 3, 1, 2000000000), (1030, 2, 256, 256, 2, 0, 70000),
    (3, 5, 256, 16, 1, 0, 4096), (1027, 7, 64, 48, 3, 0, 131072), (2, 40, 128, 96, 1, 1, 9)])
def test_rope_matches_the_reference(dtype, T, H, D, rot, axes, pairs, far):
    torch = _torch()
    rng = np.random.default_rng(T + D)
    say("rope", T, H, D, rot, axes, pairs, far, dtype)
    sections, pos, freq = _rope_inputs(rng, T, axes, rot // 2, far)
    X, x = to16(rng.standard_normal((T, H, D)) * 3, dtype)
    want = ref.rope(x, pos, freq, sections, pairs)
    bound = _rope_bound(want, x, rot // 2, pairs, dtype)
    P, F = cuda(pos), cuda(freq)
    Y = torch.full_like(X, float("nan"))
    w4.kv4_rope(X, Y, P, F, sections, pairs)
    assert (np.abs(host(Y) - want) <= bound).all()
    if rot < D:                                     # the rest is copied
        assert torch.equal(Y[..., rot:], X[..., rot:])
    # in place; heads outside tokens, padded; a wider positions tensor
    Z = X.clone()
    w4.kv4_rope(Z, Z, P, F, sections, pairs)
    assert torch.equal(Z, Y)
    wide = torch.full((H, T, D + 16), 7.0, dtype=X.dtype, device="cuda")
    view = wide[..., :D].transpose(0, 1)
    view.copy_(X)
    out = torch.full((T, H + 1, D + 8), 5.0, dtype=X.dtype, device="cuda")
    pw = torch.zeros((axes, T + 3), dtype=torch.int32, device="cuda")
    pw[:, :T] = P
    w4.kv4_rope(view, out[:, 1:, :D], pw, F, sections, pairs)
    assert torch.equal(out[:, 1:, :D], Y)
    assert bool((out[:, 0] == 5).all()) and bool((out[..., D:] == 5).all())


def test_rope_of_nothing():
    torch = _torch()
    X = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    P = torch.zeros((1, 0), dtype=torch.int32, device="cuda")
    w4.kv4_rope(X, X, P, cuda(np.ones(32)), (32,))


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _slots(rng, T, pages, page):
    s = rng.permutation(pages * page)[:T].astype(np.int32)
    s[rng.random(T) < 0.1] = -1
    if T > 3:
        s[2] = pages * page           # outside: skipped
        s[3] = -2147483648
    return s


def _special_rows(x):
    """Rows of unlike size, constant, huge, tiny and non-finite ones."""
    T = x.shape[0]
    x = x * np.exp(np.linspace(-6, 6, T))[:, None, None]
    for i, row in enumerate((0.0, 1.5, -0.0, np.nan, np.inf, -np.inf, 1e-7, 6e4)):
        if 4 + i < T:
            if np.isfinite(row):
                x[4 + i, 0] = row
            else:
                x[4 + i, 0, 3 * i] = row
    return x


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,H,D,pages,page", [
    (1, 1, 64, 1, 16), (7, 2, 128, 3, 16), (40, 3, 256, 5, 32), (300, 8, 128, 9, 64),
    (129, 5, 64, 2, 1024), (1100, 2, 64, 20, 128)])
def test_append_is_the_stored_form_bit_for_bit(dtype, T, H, D, pages, page):
    torch = _torch()
    rng = np.random.default_rng(T * D)
    say("append", T, H, D, pages, page, dtype)
    T = min(T, pages * page)
    with np.errstate(over="ignore"):
        K, k = to16(_special_rows(rng.standard_normal((T, H, D))), dtype)
        V, v = to16(_special_rows(rng.standard_normal((T, H, D)))[::-1].copy(), dtype)
    slots = _slots(rng, T, pages, page)
    cache = rng.integers(0, 256, (pages, H, page, D + 8)).astype(np.uint8)
    want = cache.copy()
    ref.store(want, slots, k, v)
    C = cuda(cache)
    w4.kv4_append(K, V, cuda(slots), C)
    # -0 and +0 offsets are the same value
    got = C.cpu().numpy()
    differ = np.flatnonzero(got.reshape(-1) != want.reshape(-1))
    assert ((got.reshape(-1)[differ] | want.reshape(-1)[differ]) == 0x80).all(), differ[:20]
    # from strided parts of one buffer
    qkv = torch.zeros((T, 3 * H + 1, D), dtype=K.dtype, device="cuda")
    qkv[:, H:2 * H] = K
    qkv[:, 2 * H:3 * H] = V
    C2 = cuda(cache)
    w4.kv4_append(qkv[:, H:2 * H], qkv[:, 2 * H:3 * H], cuda(slots), C2)
    assert torch.equal(C, C2)
    # read back, rounded once
    Ko = torch.full((T, H, D), 3.0, dtype=K.dtype, device="cuda")
    Vo = torch.full_like(Ko, 3.0)
    w4.kv4_dequant_debug(cuda(slots), C, Ko, Vo)
    for out, part in zip((Ko, Vo), ref.load(got, slots)):
        # exact product, sum rounded to FP32, then to 16 bits
        c, s, z = (x.astype(np.float32) for x in part)
        with np.errstate(invalid="ignore"):
            exact = torch.from_numpy(c * s[..., None] + z[..., None]).to(K.dtype)
        assert torch.equal(out.cpu().nan_to_num(9.0), exact.nan_to_num(9.0))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,Hq,H,D,rot,axes,pairs", [
    (1, 8, 2, 128, 128, 1, 0), (33, 3, 3, 64, 32, 2, 1), (1025, 4, 1, 128, 128, 3, 0),
    (50, 0, 2, 256, 256, 3, 0), (9, 16, 1, 256, 192, 1, 1)])
def test_rope_append_stores_rotated_keys(dtype, T, Hq, H, D, rot, axes, pairs):
    torch = _torch()
    rng = np.random.default_rng(T + rot)
    pages, page = T // 32 + 2, 32
    say("rope_append", T, Hq, H, D, rot, axes, pairs, dtype)
    sections, pos, freq = _rope_inputs(rng, T, axes, rot // 2, 50000)
    qkv, x = to16(rng.standard_normal((T, Hq + 2 * H, D)), dtype)
    Q, K, V = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    k = x[:, Hq:Hq + H]
    slots = _slots(rng, T, pages, page)
    S, P, F = cuda(slots), cuda(pos), cuda(freq)
    C = torch.zeros((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
    Qo = torch.empty((T, Hq, D), dtype=qkv.dtype, device="cuda") if Hq else None
    before = qkv.clone()
    w4.kv4_rope_append(Q if Hq else None, K, V, Qo, P, F, sections, pairs, S, C)
    assert torch.equal(qkv, before)
    if Hq:
        Y = torch.empty_like(Qo)
        w4.kv4_rope(Q, Y, P, F, sections, pairs)
        assert torch.equal(Y, Qo)
        w4.kv4_rope_append(Q, K, V, Q, P, F, sections, pairs, S, C.clone())
        assert torch.equal(Q, Y)
    turned = ref.rope(k, pos, freq, sections, pairs)
    (kc, ks, kz), part_v = ref.load(C.cpu().numpy(), slots)
    there = (slots >= 0) & (slots < pages * page)
    # half a step; the end codes add the roundings of scale (15/2 steps of
    # 2^-11) and offset; the rotation its FP32 error
    got = kc * ks[..., None] + kz[..., None]
    bound = (0.5 + 16 * 2.0 ** -11) * ks[..., None] + 2.0 ** -10 * np.abs(kz[..., None]) \
        + _rope_bound(turned, k, rot // 2, pairs, "float32")
    assert (np.abs(got - turned) <= bound)[there].all()
    # values are stored as kv4_append stores them
    C2 = torch.zeros_like(C)
    w4.kv4_append(K, V, S, C2)
    for a, b in zip(part_v, ref.load(C2.cpu().numpy(), slots)[1]):
        assert (a == b).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def _filled(rng, pages, H, page, D, spread=1.0):
    """A cache whose every slot was appended to by the library."""
    torch = _torch()
    n = pages * page
    k = rng.standard_normal((n, H, D)) * np.exp(rng.standard_normal((1, H, D)) * 0.4)
    v = rng.standard_normal((n, H, D)) * np.exp(rng.standard_normal((n, H, 1)) * spread)
    C = torch.empty((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
    K, V = (torch.from_numpy(x.astype(np.float32)).half().cuda() for x in (k, v))
    w4.kv4_append(K, V, torch.arange(n, dtype=torch.int32, device="cuda"), C)
    return C


def _check(o, lse, expect, name, keys, what=""):
    want, want_lse, weight, size, floor, reach = expect
    rows = ~np.isnan(want_lse)
    score = 8 * U * reach
    step = 2.0 ** -11 if name == "bfloat16" else 2.0 ** -21
    bound = (half_eps(name) * np.abs(want) + 2.0 ** -25 * (1 + floor) + step * weight
             + (2 * score[..., None] + (64 + keys / 32) * U) * size)
    err = np.abs(host(o) - want)
    assert (err <= bound)[rows].all(), (what, float((err / bound)[rows].max()))
    if lse is not None:
        got = lse.double().cpu().numpy()
        empty = np.isneginf(want_lse)
        assert np.isneginf(got[empty]).all(), what
        ok = rows & ~empty
        tol = score + 64 * U * (1 + np.abs(want_lse))
        assert (np.abs(got[ok] - want_lse[ok]) <= tol[ok]).all(), what


def _attend(q, C, table, lens, starts, Hq, scale, window, max_q, max_len, lse=True, T=None):
    """(O, lse) on device tensors; rows of no request keep 9."""
    torch = _torch()
    B, H, D = table.shape[0], C.shape[1], C.shape[3] - 8
    O = torch.full_like(q, 9.0)
    L = torch.full(q.shape[:2], 9.0, dtype=torch.float32, device="cuda") if lse else None
    ws = w4.alloc_kv4_workspace(B, Hq, H, D, max_q, max_len, window)
    w4.kv4_attention(q, C, cuda(np.asarray(table, np.int32)), cuda(np.asarray(lens, np.int32)),
                     None if starts is None else cuda(np.asarray(starts, np.int32)), O, L, scale,
                     window, max_q, max_len, ws)
    torch.cuda.synchronize()
    if ws is not None:                              # ready for the next call
        assert int(ws[:65536].sum()) == 0
    return O, L


def _requests(rng, lens, pages, page):
    width = max(1, -(-max(lens) // page)) + 1
    ids = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        used = -(-n // page)
        table[b, :used] = ids[at: at + used]
        at += used
    assert at <= pages
    return table


ATTENTION = [
    # D, Hq, H, page, lens, new tokens, window
    (128, 4, 4, 16, [1, 0, 15, 16, 17, 31, 33, 200], [1] * 8, 0),
    (64, 8, 2, 32, [1, 64, 65, 130], [1, 3, 0, 5], 0),
    (128, 8, 1, 64, [63, 64, 257], [2, 1, 4], 0),
    (256, 6, 2, 16, [5, 40, 100], [1, 2, 7], 0),
    (128, 16, 1, 16, [90], [1], 0),
    (128, 20, 1, 16, [90, 7], [1, 1], 0),             # more than 16 rows
    (64, 7, 7, 128, [300, 12], [1, 1], 50),           # window
    (128, 8, 2, 16, [70, 100, 33], [3, 40, 33], 17),  # rows and window
    (128, 3, 1, 16, [2, 4], [5, 9], 0),               # more queries than tokens: empty rows
    (64, 4, 2, 64, [150], [150], 0),                  # a whole prompt
    (128, 4, 4, 32, [129, 64], [100, 64], 0),
    (256, 2, 1, 32, [77], [70], 33),
    (128, 28, 4, 16, [50, 60, 1], [11, 12, 1], 0),
    (64, 1, 1, 16, [1], [1], 1),
]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention_matches_the_reference(dtype, case):
    D, Hq, H, page, lens, new, window = ATTENTION[case]
    rng = np.random.default_rng(case)
    say("attention", dtype, *ATTENTION[case])
    pages = sum(-(-n // page) for n in lens) + 2
    C = _filled(rng, pages, H, page, D)
    table = _requests(rng, lens, pages, page)
    starts = np.concatenate(([0], np.cumsum(new)))
    T = int(starts[-1]) + 3                           # rows that no request has
    Q, q = to16(rng.standard_normal((T, Hq, D)) * 1.5, dtype)
    scale = D ** -0.5
    O, L = _attend(Q, C, table, lens, starts, Hq, scale, window, max(new), max(lens))
    expect = ref.attention(q, C.cpu().numpy(), table, lens, starts, scale, window)
    _check(O, L, expect, dtype, max(lens), ATTENTION[case])
    assert bool((O[-3:] == 9).all()) and bool((L[-3:] == 9).all())
    # planned for other lengths, without lse: the same rows
    for planned in (0, 16 * max(lens)):
        O2, _ = _attend(Q, C, table, lens, starts, Hq, scale, window, max(new), planned,
                        lse=False)
        _check(O2, None, expect, dtype, max(lens), (planned, *ATTENTION[case]))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_attention_one_query_per_request_without_starts(dtype):
    torch = _torch()
    rng = np.random.default_rng(20)
    lens, page, H, Hq, D = [40, 0, 17, 5], 16, 2, 6, 64
    C = _filled(rng, 9, H, page, D)
    table = _requests(rng, lens, 9, page)
    Q, q = to16(rng.standard_normal((4, Hq, D)), dtype)
    O, L = _attend(Q, C, table, lens, None, Hq, 0.2, 0, 1, 40)
    _check(O, L, ref.attention(q, C.cpu().numpy(), table, lens, None, 0.2), dtype, 40)
    O2, L2 = _attend(Q, C, table, lens, [0, 1, 2, 3, 4], Hq, 0.2, 0, 1, 40)
    assert torch.equal(O, O2) and torch.equal(L, L2)


def test_attention_never_sees_masked_places():
    """NaN and infinite parameters and any codes beyond the length, in pages
    of others and in entries that are no pages, change nothing."""
    torch = _torch()
    rng = np.random.default_rng(21)
    for D, page, lens, new, window in ((128, 16, [37, 70, 5], [1, 3, 1], 0),
                                       (64, 64, [100, 3, 65], [90, 1, 65], 0),
                                       (128, 32, [300, 40, 41], [2, 2, 2], 33)):
        H, Hq, pages = 2, 8, 40
        C = _filled(rng, pages, H, page, D)
        table = _requests(rng, lens, pages, page)
        starts = np.concatenate(([0], np.cumsum(new)))
        Q, q = to16(rng.standard_normal((int(starts[-1]), Hq, D)), "float16")
        O, L = _attend(Q, C, table, lens, starts, Hq, 0.1, window, max(new), max(lens))
        held = np.zeros((pages, page), bool)
        for b, n in enumerate(lens):
            j = np.arange(max(0, n - new[b] - window + 1) if window else 0, n)
            held[table[b, j // page], j % page] = True
        for fill in (0x7E7E, 0x7C00, 0xFC00, 0xFFFF):
            D2 = C.cpu().numpy()
            flat = D2.reshape(-1)
            for p in range(pages):
                for at in np.flatnonzero(~held[p]):
                    for h in range(H):
                        base, r = ref._unit(pages, H, page, D, p * page + at, h)
                        for off in (16 * D, 16 * D + 64):
                            flat[base + off + 4 * r: base + off + 4 * r + 4] = \
                                np.array([fill, fill], "<u2").view(np.uint8)
                        flat[base + r * (D // 2): base + (r + 1) * (D // 2)] = 0xFF
            wild = table.copy()
            wild[wild < 0] = rng.choice([-1, pages, 2147483647, -2147483648, 0],
                                        (wild < 0).sum())
            O2, L2 = _attend(Q, cuda(D2), wild, lens, starts, Hq, 0.1, window, max(new),
                             max(lens))
            assert torch.equal(O, O2) and torch.equal(L, L2), hex(fill)


def test_a_stored_nan_reaches_the_queries_that_see_it_only():
    """A token stored with an infinite key or a NaN value: queries before it,
    and those whose window has passed it, are as without it."""
    torch = _torch()
    rng = np.random.default_rng(29)
    for D, n, window, bad_key in ((128, 150, 0, False), (64, 150, 40, True), (128, 90, 20, False)):
        H, Hq, page, pages = 1, 4, 16, 12
        C = _filled(rng, pages, H, page, D)
        table = _requests(rng, [n], pages, page)
        Q, q = to16(rng.standard_normal((n, Hq, D)), "float16")
        O, L = _attend(Q, C, table, [n], [0, n], Hq, 0.1, window, n, n)
        at = 45
        slot = int(table[0, at // page]) * page + at % page
        kv = torch.randn((2, 1, H, D), device="cuda").half()
        kv[0 if bad_key else 1, 0, 0, 5] = float("inf" if bad_key else "nan")
        w4.kv4_append(kv[0], kv[1], cuda(np.array([slot], np.int32)), C)
        O2, L2 = _attend(Q, C, table, [n], [0, n], Hq, 0.1, window, n, n)
        sees = np.arange(n) >= at
        if window:
            sees &= np.arange(n) < at + window
        sees = torch.from_numpy(sees)
        assert torch.equal(O[~sees], O2[~sees]) and torch.equal(L[~sees], L2[~sees])
        assert bool(O2[sees].isnan().all())


def test_attention_treats_bad_pages_as_not_there():
    rng = np.random.default_rng(22)
    page, H, Hq, D, pages = 16, 1, 4, 128, 14
    C = _filled(rng, pages, H, page, D)
    lens, new = [100, 50, 20], [1, 30, 2]
    table = _requests(rng, lens, pages, page)
    table[0, 1], table[0, 4], table[1, 0], table[2, :] = -1, pages, 1 << 30, -7
    starts = np.concatenate(([0], np.cumsum(new)))
    Q, q = to16(rng.standard_normal((33, Hq, D)), "float16")
    O, L = _attend(Q, C, table, lens, starts, Hq, 0.1, 0, 30, 100)
    _check(O, L, ref.attention(q, C.cpu().numpy(), table, lens, starts, 0.1), "float16", 100)


def test_attention_split_and_unsplit_lengths():
    """One request cut into many token ranges, lengths around the cuts."""
    rng = np.random.default_rng(23)
    page, H, Hq, D = 64, 1, 2, 64
    n = 5000
    pages = -(-n // page)
    C = _filled(rng, pages, H, page, D, spread=2.0)
    host_c = C.cpu().numpy()
    Q, q = to16(rng.standard_normal((3, Hq, D)) * 2, "float16")
    for length in (5000, 4097, 4096, 4095, 300, 257, 256, 129, 31):
        table = _requests(rng, [length], pages, page)
        for planned in (5000, length, 64):
            say("split", length, planned, w4.kv4_attention_describe(1, Hq, H, D, 3, planned))
            O, L = _attend(Q, C, table, [length], [0, 3], Hq, 0.125, 0, 3, planned)
            expect = ref.attention(q, host_c, table, [length], [0, 3], 0.125)
            _check(O, L, expect, "float16", length, (length, planned))


def test_attention_values_of_every_size():
    """Scales over FP16's whole range in one sequence, zero scales (constant
    values), one key that takes all the weight, and BF16 queries of any size."""
    torch = _torch()
    rng = np.random.default_rng(24)
    page, H, Hq, D, n = 16, 1, 4, 128, 700
    pages = -(-n // page)
    table = np.arange(pages, dtype=np.int32)[None]
    for kind in range(5):
        k = rng.standard_normal((n, H, D)).astype(np.float32)
        v = rng.standard_normal((n, H, D)).astype(np.float32)
        qs = rng.standard_normal((2, Hq, D)).astype(np.float32)
        if kind == 0:
            v *= np.exp2(np.linspace(-20, 12, n))[:, None, None]
        elif kind == 1:
            v *= np.exp2(np.linspace(12, -20, n))[:, None, None]
        elif kind == 2:
            v[::2] = 0.75                           # scale 0
            v[:64] = 0
        elif kind == 3:
            k[401] = 4 * qs[0, 0] * np.sign(1)      # one logit far above the rest
        else:
            qs *= np.exp2(np.array([-120.0, -40, 3, 0]))[None, :, None]
        name = "bfloat16" if kind == 4 else "float16"
        K, V = (torch.from_numpy(x).half().cuda() for x in (k, v))
        C = torch.empty((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
        w4.kv4_append(K, V, torch.arange(n, dtype=torch.int32, device="cuda"), C)
        Q, q = to16(qs, name)
        O, L = _attend(Q, C, table, [n], [0, 2], Hq, 0.5, 0, 2, n)
        expect = ref.attention(q, C.cpu().numpy(), table, [n], [0, 2], 0.5)
        _check(O, L, expect, name, n, kind)


def test_attention_of_strided_queries_and_outputs():
    torch = _torch()
    rng = np.random.default_rng(25)
    lens, new, page, H, Hq, D = [50, 33], [2, 20], 16, 2, 4, 128
    C = _filled(rng, 8, H, page, D)
    table = _requests(rng, lens, 8, page)
    qkv = torch.randn((22, Hq + 2 * H, D), device="cuda").half()
    Q = qkv[:, :Hq]
    a, la = _attend(Q.contiguous(), C, table, lens, [0, 2, 22], Hq, 0.1, 0, 20, 50)
    O = torch.full((Hq, 22, D + 8), 4.0, dtype=torch.float16, device="cuda")
    L = torch.empty((22, Hq), device="cuda")
    ws = w4.alloc_kv4_workspace(2, Hq, H, D, 20, 50)
    w4.kv4_attention(Q, C, cuda(table), cuda(np.array(lens, np.int32)),
                     cuda(np.array([0, 2, 22], np.int32)), O[..., :D].transpose(0, 1), L, 0.1, 0,
                     20, 50, ws)
    assert torch.equal(O[..., :D].transpose(0, 1), a) and torch.equal(L, la)
    assert bool((O[..., D:] == 4).all())


def test_attention_past_four_gigabytes():
    """Pages at both ends of a cache whose byte offsets pass 32 bits."""
    torch = _torch()
    rng = np.random.default_rng(26)
    page, H, Hq, D = 64, 8, 8, 128
    pages = (5 << 30) // (H * page * (D + 8))
    C = torch.empty((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
    small = _filled(rng, 4, H, page, D)
    table = np.array([[0, pages - 1, pages // 2, pages - 2]], np.int32)
    lens = [250]
    Q, q = to16(rng.standard_normal((1, Hq, D)), "float16")
    slots = (table[0, :, None].astype(np.int64) * page + np.arange(page)).reshape(-1)
    K = torch.empty((256, H, D), dtype=torch.float16, device="cuda")
    V = torch.empty_like(K)
    w4.kv4_dequant_debug(torch.arange(256, dtype=torch.int32, device="cuda"), small, K, V)
    w4.kv4_append(K, V, cuda(slots.astype(np.int32)), C)
    again = torch.empty_like(small)
    w4.kv4_append(K, V, torch.arange(256, dtype=torch.int32, device="cuda"), again)
    for i, p in enumerate(table[0]):
        assert torch.equal(C[p], again[i])
    O, L = _attend(Q, C, table, lens, [0, 1], Hq, 0.1, 0, 1, 250)
    O2, L2 = _attend(Q, again, np.arange(4, dtype=np.int32)[None], lens, [0, 1], Hq, 0.1, 0, 1,
                     250)
    assert torch.equal(O, O2) and torch.equal(L, L2)


def test_a_decode_step_on_another_stream_and_in_a_graph():
    """tables -> rope and append -> attention: eager on a side stream, and
    replayed from a graph with eager work between the replays, give the same
    bits; lengths grow inside the graph."""
    torch = _torch()
    rng = np.random.default_rng(27)
    B, page, width, H, Hq, D = 5, 16, 40, 2, 8, 128
    pages = B * width
    cache0 = _filled(rng, pages, H, page, D)
    i32 = dict(dtype=torch.int32, device="cuda")
    start = np.array([0, 1, 300, 511, 32], np.int32)
    freq = cuda(10000.0 ** (-np.arange(D // 2) / (D // 2)))
    ws = w4.alloc_kv4_workspace(B, Hq, H, D, 1, 600)
    assert ws is not None
    steps = [torch.randn((B, Hq + 2 * H, D), device="cuda").half() for _ in range(6)]

    def state():
        table, ring, st = w4.alloc_kv4_pages(pages, B, width)
        lens, zero = torch.zeros(B, **i32), torch.zeros(B + 1, **i32)
        big = torch.zeros(1024, **i32)
        w4.kv4_tables(lens, cuda(start), table, ring, st, lens, st, zero, big, big.clone(), page)
        return dict(cache=cache0.clone(), table=table, ring=ring, st=st, lens=lens,
                    want=torch.zeros(B, **i32), starts=torch.zeros(B + 1, **i32),
                    slots=torch.zeros(B, **i32), pos=torch.zeros(B, **i32),
                    qkv=torch.zeros((B, Hq + 2 * H, D), dtype=torch.float16, device="cuda"),
                    O=torch.zeros((B, Hq, D), dtype=torch.float16, device="cuda"),
                    L=torch.zeros((B, Hq), device="cuda"))

    def step(s, stream=None):
        w4.kv4_tables(s["lens"], s["want"], s["table"], s["ring"], s["st"], s["lens"], s["st"],
                      s["starts"], s["slots"], s["pos"], page, stream)
        q, k, v = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + H], s["qkv"][:, Hq + H:]
        w4.kv4_rope_append(q, k, v, q, s["pos"], freq, (D // 2,), 0, s["slots"], s["cache"],
                           stream)
        w4.kv4_attention(q, s["cache"], s["table"], s["lens"], s["starts"], s["O"], s["L"], 0.09,
                         0, 1, 600, ws, stream)

    a, b = state(), state()
    torch.cuda.synchronize()
    side, eager = torch.cuda.Stream(), []
    for x in steps:
        a["qkv"].copy_(x)
        a["want"].copy_(a["lens"] + 1)
        side.wait_stream(torch.cuda.current_stream())
        step(a, side)
        torch.cuda.current_stream().wait_stream(side)
        eager.append((a["O"].clone(), a["L"].clone()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for i, x in enumerate(steps):
        b["qkv"].copy_(x)
        b["want"].copy_(b["lens"] + 1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["O"], eager[i][0]) and torch.equal(b["L"], eager[i][1]), i
        torch.randn(1 << 20, device="cuda").sum()
    assert b["lens"].tolist() == (start + 6).tolist()
    assert torch.equal(a["cache"], b["cache"]) and torch.equal(a["table"], b["table"])


def test_results_repeat_bit_for_bit():
    """Splits joined by whichever workgroup comes last, in a fixed order; one
    workspace for calls of unlike shapes in turn."""
    torch = _torch()
    rng = np.random.default_rng(28)
    page, H, Hq, D = 32, 2, 8, 128
    C = _filled(rng, 130, H, page, D)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    runs = []
    for lens, new in (([4000], [1]), ([1000, 2000, 700], [1, 2, 1])):
        table = cuda(_requests(rng, lens, 130, page))
        starts = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
        runs.append((torch.randn((int(starts[-1]), Hq, D), device="cuda").half(), table,
                     cuda(np.array(lens, np.int32)), cuda(starts), max(new), max(lens)))
    first = [None, None]
    for _ in range(20):
        for i, (Q, table, lens, starts, mq, ml) in enumerate(runs):
            O, L = torch.empty_like(Q), torch.empty(Q.shape[:2], device="cuda")
            w4.kv4_attention(Q, C, table, lens, starts, O, L, 0.1, 0, mq, ml, ws)
            if first[i] is None:
                first[i] = (O, L)
            assert torch.equal(O, first[i][0]) and torch.equal(L, first[i][1])


def test_binding_refuses_on_the_device():
    torch = _torch()
    C = w4.alloc_kv4_cache(4, 2, 64, 16)
    Q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    O = torch.zeros_like(Q)
    t = torch.zeros((2, 200), dtype=torch.int32, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert w4.kv4_attention_workspace_bytes(2, 4, 2, 64, 1, 3000) > 0
    with pytest.raises(w4.W4A16Error) as e:
        w4.kv4_attention(Q, C, t, n, None, O, None, 0.1, 0, 1, 3000, None)
    assert e.value.name == "W4A16_ERR_WORKSPACE"
    with pytest.raises(ValueError, match="workspace"):
        w4.kv4_attention(Q, C, t, n, None, O, None, 0.1, 0, 1, 3000,
                         torch.zeros(1024, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="heads|expected"):
        w4.kv4_append(Q, Q, n, C)
    with pytest.raises(ValueError, match="channels must be contiguous"):
        w4.kv4_rope(Q.transpose(1, 2), O.transpose(1, 2), n[None], cuda(np.ones(32)), (32,))
    with pytest.raises(w4.W4A16Error):
        w4.kv4_rope(Q[..., :32], O[..., :32], n[None], cuda(np.ones(16)), (16,))
    with pytest.raises(ValueError, match="rows for"):
        w4.kv4_attention(Q[:1], C, t, n, None, O[:1], None, 0.1, 0, 1, 30, None)
    torch.cuda.synchronize()
