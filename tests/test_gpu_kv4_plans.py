"""kv4_attention through both kernels and in token ranges: the plan follows
from the sizes a call is planned for, which may be more than it then holds.

Tolerances as for the other attention tests: the output's rounding, the
rounding of each weight to FP16 (2^-11; FP16 calls carry the remainder:
2^-21), half of FP16's smallest step at the largest weight, eight roundings
of the largest magnitude in a score, and sums of n terms in FP32 taken as
64 + n/32 roundings of the sum of magnitudes.
"""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import kv4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CUS = 256


def _inputs(rng, lens, new, page, Hq, H, D, dtype):
    import torch
    T, pages = sum(new), sum(-(-n // page) for n in lens) + 3
    k = rng.standard_normal((pages * page, H, D)) * np.exp(rng.standard_normal((1, H, D)) * 0.3)
    v = rng.standard_normal((pages * page, H, D)) * np.exp(
        rng.standard_normal((pages * page, H, 1)) * 0.7)
    cache = torch.empty((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
    K, V = (torch.from_numpy(x.astype(np.float32)).half().cuda() for x in (k, v))
    w4.kv4_append(K, V, torch.arange(pages * page, dtype=torch.int32, device="cuda"), cache)
    ids, at = rng.permutation(pages), 0
    table = np.full((len(lens), max(-(-n // page) for n in lens) + 1), -1, np.int32)
    for b, n in enumerate(lens):
        used = -(-n // page)
        table[b, :used] = ids[at:at + used]
        at += used
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((T, Hq, D)).astype(np.float32)).to(
        getattr(torch, dtype)).cuda()
    return q, cache, table, starts


def _reference(q, cache, table, lens, starts, scale, window):
    """(o, lse, bound without the output's rounding) in 64 bits, by head."""
    pages, H, page, d8 = cache.shape
    T, Hq, D = q.shape
    q = q.double().cpu().numpy()
    host = cache.cpu().numpy()
    o, lse = np.zeros(q.shape), np.full((T, Hq), -np.inf)
    weight, size, floor = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    reach = np.zeros((T, Hq))
    for b, n in enumerate(lens):
        t0, t1 = int(starts[b]), int(starts[b + 1])
        if t0 == t1 or n == 0:
            continue
        j = np.arange(n)
        slots = table[b, j // page].astype(np.int64) * page + j % page
        (kc, ks, kz), (vc, vs, vz) = ref.load(host, slots)
        pos = n - (t1 - t0) + np.arange(t1 - t0)
        hide = j[None] > pos[:, None]
        if window:
            hide |= j[None] <= pos[:, None] - window
        for h in range(Hq):
            g = h // (Hq // H)
            k, v = (c[:, g] * s[:, g, None] + z[:, g, None]
                    for c, s, z in ((kc, ks, kz), (vc, vs, vz)))
            x = scale * (q[t0:t1, h] @ k.T)
            x[hide] = -np.inf
            m = x.max(1, keepdims=True)
            m[np.isneginf(m)] = 0
            p = np.exp(x - m)
            total = p.sum(1, keepdims=True)
            some = total[:, 0] > 0
            p[some] /= total[some]
            lse[t0:t1, h][some] = (m + np.log(np.where(total > 0, total, 1)))[some, 0]
            o[t0:t1, h] = p @ v
            weight[t0:t1, h] = p @ (vs[:, g, None] * np.abs(vc[:, g]))
            size[t0:t1, h] = (p @ (15 * vs[:, g] + np.abs(vz[:, g])))[:, None]
            floor[t0:t1, h] = 8 * n * (p * vs[:, g]).max(1)[:, None]
            reach[t0:t1, h] = (scale * np.abs(q[t0:t1, h]).sum(1)
                               * (23 * ks[:, g] + np.abs(kz[:, g])).max())
    return o, lse, weight, size, floor, reach


# D, Hq, H, page, lens, new tokens, window, planned (B, queries, tokens), kernel, ranges
CASES = [
    (128, 4, 4, 32, [129, 64], [100, 64], 0, (16384, 16384), "rows", False),
    (128, 24, 8, 16, [333, 20, 1, 90], [26, 20, 1, 30], 0, (1024, 8192), "rows", False),
    (64, 4, 2, 64, [150, 3], [150, 5], 0, (16384, 16384), "rows", False),
    (64, 6, 1, 16, [700, 40], [70, 33], 65, (65536, 65536), "rows", False),
    (256, 2, 1, 32, [77, 200], [70, 1], 33, (16384, 16384), "rows", False),
    (256, 3, 1, 256, [300, 10], [90, 10], 0, (1024, 65536), "rows", False),
    (128, 8, 1, 64, [3500], [33], 0, (2048, 6000), "rows", True),
    (64, 8, 1, 16, [2500], [40], 0, (2048, 4000), "rows", True),
    (256, 8, 1, 128, [2600], [20], 0, (2048, 1500), "rows", True),
    (256, 8, 1, 16, [1000], [33], 0, (2048, 1500), "rows", True),
    (128, 8, 1, 16, [2100], [300], 700, (300, 2100), None, False),
    (128, 5, 1, 32, [1000, 70], [18, 40], 0, (40, 1000), "tokens", True),
    (64, 3, 1, 16, [900, 33, 0], [21, 3, 2], 0, (21, 900), "tokens", True),
    (256, 9, 1, 64, [700], [2], 0, (2, 700), "tokens", True),
    (256, 4, 2, 16, [900, 50], [3, 4], 100, (4, 120), "tokens", False),
    (64, 4, 1, 32, [2500, 1, 31], [2, 1, 2], 0, (2, 2500), "tokens", True),
    (128, 1, 1, 16, [4000], [8], 0, (8, 4000), "tokens", True),
]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_through_every_kernel(dtype, case):
    import torch
    D, Hq, H, page, lens, new, window, (max_q, max_len), kernel, ranges = CASES[case]
    text = w4.kv4_attention_describe(len(lens), Hq, H, D, max_q, max_len, window, 0)
    say("attention plan", dtype, *CASES[case], text)
    rng = np.random.default_rng(100 + case)
    q, cache, table, starts = _inputs(rng, lens, new, page, Hq, H, D, dtype)
    O = torch.full_like(q, 9.0)
    L = torch.full(q.shape[:2], 9.0, device="cuda")
    ws = w4.alloc_kv4_workspace(len(lens), Hq, H, D, max_q, max_len, window)
    i32 = dict(dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    args = (torch.tensor(table, **i32), torch.tensor(lens, **i32), torch.tensor(starts, **i32))
    for _ in range(2):
        w4.kv4_attention(q, cache, *args, O, L, scale, window, max_q, max_len, ws)
    torch.cuda.synchronize()
    if ws is not None:
        assert int(ws[:65536].sum()) == 0
    want, lse, weight, size, floor, reach = _reference(q, cache, table, lens, starts, scale, window)
    n, eps = max(lens), torch.finfo(q.dtype).eps / 2
    step = 2.0 ** -11 if dtype == "bfloat16" else 2.0 ** -21
    bound = (eps * np.abs(want) + 2.0 ** -25 * (1 + floor) + step * weight
             + (16 * U * reach[..., None] + (64 + n / 32) * U) * size)
    err = np.abs(O.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / bound).max())
    got = L.double().cpu().numpy()
    empty = np.isneginf(lse)
    assert np.isneginf(got[empty]).all()
    tol = 8 * U * reach[~empty] + 64 * U * (1 + np.abs(lse[~empty]))
    assert (np.abs(got[~empty] - lse[~empty]) <= tol).all()


@pytest.mark.parametrize("case", range(len(CASES)))
def test_what_no_query_sees_reaches_no_result(case):
    """NaN in every place that is masked for all queries, in either kernel,
    changes no bit; nor does a workspace another plan has used."""
    import torch
    D, Hq, H, page, lens, new, window, (max_q, max_len), kernel, ranges = CASES[case]
    say("attention masked", *CASES[case])
    rng = np.random.default_rng(300 + case)
    q, cache, table, starts = _inputs(rng, lens, new, page, Hq, H, D, "float16")
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (torch.tensor(table, **i32), torch.tensor(lens, **i32), torch.tensor(starts, **i32))
    nbytes = max(w4.kv4_attention_workspace_bytes(len(lens), Hq, H, D, mq, ml, window)
                 for mq, ml in ((max_q, max_len), (max(new), max(lens) + 1)))
    ws = torch.zeros(nbytes + 16, dtype=torch.uint8, device="cuda")

    def run(mq, ml):
        O, L = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
        w4.kv4_attention(q, cache, *args, O, L, D ** -0.5, window, mq, ml, ws)
        torch.cuda.synchronize()
        return O, L

    before = run(max_q, max_len)
    other = run(max(new), max(lens) + 1)            # the plan of the sizes as they are
    seen = np.zeros(cache.shape[0] * page, bool)
    for b, n in enumerate(lens):
        first = max(0, n - new[b] - window + 1) if window else 0
        j = np.arange(first, n)
        if new[b]:
            seen[table[b, j // page].astype(np.int64) * page + j % page] = True
    bad = torch.from_numpy(np.flatnonzero(~seen).astype(np.int32)).cuda()
    assert bad.numel() > 0
    K = torch.full((bad.numel(), H, D), float("nan"), dtype=torch.float16, device="cuda")
    w4.kv4_append(K, K, bad, cache)
    for then, now in zip((*before, *other), (*run(max_q, max_len), *run(max(new), max(lens) + 1))):
        assert torch.isfinite(then.float()).all() or (lens[-1] < new[-1])
        assert torch.equal(then, now)


@pytest.mark.parametrize("case", [i for i, c in enumerate(CASES) if max(c[5]) > 1])
def test_a_stored_nan_stays_with_the_queries_that_see_it(case):
    """The last token of every request that has several queries is NaN: its
    last query is, the others are within the reference's bounds as before."""
    import torch
    D, Hq, H, page, lens, new, window, (max_q, max_len), kernel, ranges = CASES[case]
    say("attention nan", *CASES[case])
    rng = np.random.default_rng(400 + case)
    q, cache, table, starts = _inputs(rng, lens, new, page, Hq, H, D, "bfloat16")
    scale, n = D ** -0.5, max(lens)
    want, lse, weight, size, floor, reach = _reference(q, cache, table, lens, starts, scale, window)
    last = [b for b in range(len(lens)) if new[b] > 1 and lens[b] >= 1]
    slots = torch.tensor([int(table[b, (lens[b] - 1) // page]) * page + (lens[b] - 1) % page
                          for b in last], dtype=torch.int32, device="cuda")
    K = torch.full((len(last), H, D), float("nan"), dtype=torch.float16, device="cuda")
    w4.kv4_append(K, K, slots, cache)
    i32 = dict(dtype=torch.int32, device="cuda")
    O, L = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    w4.kv4_attention(q, cache, torch.tensor(table, **i32), torch.tensor(lens, **i32),
                     torch.tensor(starts, **i32), O, L, scale, window, max_q, max_len,
                     w4.alloc_kv4_workspace(len(lens), Hq, H, D, max_q, max_len, window))
    torch.cuda.synchronize()
    got = O.double().cpu().numpy()
    hit = [int(starts[b + 1]) - 1 for b in last]
    assert np.isnan(got[hit]).all() and np.isnan(L.cpu().numpy()[hit]).all()
    rest = np.setdiff1d(np.arange(q.shape[0]), hit)
    bound = (2.0 ** -8 * np.abs(want) + 2.0 ** -25 * (1 + floor) + 2.0 ** -11 * weight
             + (16 * U * reach[..., None] + (64 + n / 32) * U) * size)
    assert (np.abs(got - want) <= bound)[rest].all()


@pytest.mark.parametrize("queries,planned", [(1, 1), (5, 5), (40, 2048)])
@pytest.mark.parametrize("kind", range(5))
def test_attention_of_values_of_every_size(kind, queries, planned):
    """8 heads on one, so 8, 40 and 320 rows: each kernel.  Value scales over
    FP16's whole range in one sequence, rising and falling; constant values
    (scale 0); one key that takes all the weight; BF16 queries of any size."""
    import torch
    rng = np.random.default_rng(500 + kind)
    page, H, Hq, D, n = 16, 1, 8, 128, 700
    pages = -(-n // page)
    table = np.arange(pages, dtype=np.int32)[None]
    k = rng.standard_normal((n, H, D)).astype(np.float32)
    v = rng.standard_normal((n, H, D)).astype(np.float32)
    qs = rng.standard_normal((queries, Hq, D)).astype(np.float32)
    if kind == 0:
        v *= np.exp2(np.linspace(-20, 12, n))[:, None, None].astype(np.float32)
    elif kind == 1:
        v *= np.exp2(np.linspace(12, -20, n))[:, None, None].astype(np.float32)
    elif kind == 2:
        v[::2] = 0.75
        v[:64] = 0
    elif kind == 3:
        k[401] = 4 * qs[0, 0]
    else:
        qs *= np.exp2(np.array([-120.0, -40, 3, 0, -7, -1, 2, -80]))[None, :, None]
    dtype = "bfloat16" if kind == 4 else "float16"
    max_len = 6000 if planned > queries else n
    text = w4.kv4_attention_describe(1, Hq, H, D, planned, max_len, 0, CUS)
    say("attention sizes", kind, queries, text)
    assert f"<128,{8 if queries == 1 else 16 if queries == 5 else 128}," in text
    cache = torch.empty((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
    K, V = (torch.from_numpy(x).half().cuda() for x in (k, v))
    w4.kv4_append(K, V, torch.arange(n, dtype=torch.int32, device="cuda"), cache)
    q = torch.from_numpy(qs.astype(np.float32)).to(getattr(torch, dtype)).cuda()
    starts, i32 = np.array([0, queries]), dict(dtype=torch.int32, device="cuda")
    O, L = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    w4.kv4_attention(q, cache, torch.tensor(table, **i32), torch.tensor([n], **i32),
                     torch.tensor(starts, **i32), O, L, 0.5, 0, planned, max_len,
                     w4.alloc_kv4_workspace(1, Hq, H, D, planned, max_len))
    torch.cuda.synchronize()
    want, lse, weight, size, floor, reach = _reference(q, cache, table, [n], starts, 0.5, 0)
    # scores are summed among those of a workgroup: 2^-30 of the largest
    reach = np.maximum(reach, 2.0 ** -6 * reach.max())
    step = 2.0 ** -11 if dtype == "bfloat16" else 2.0 ** -21
    bound = (torch.finfo(q.dtype).eps / 2 * np.abs(want) + 2.0 ** -25 * (1 + floor)
             + step * weight + (16 * U * reach[..., None] + (64 + n / 32) * U) * size)
    err = np.abs(O.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / bound).max())
    tol = 8 * U * reach + 64 * U * (1 + np.abs(lse))
    assert (np.abs(L.double().cpu().numpy() - lse) <= tol).all()


def test_the_cases_reach_what_they_name():
    """On the device they were chosen for."""
    import torch
    if torch.cuda.get_device_properties(0).multi_processor_count != CUS:
        pytest.skip("plans depend on the number of compute units")
    seen = set()
    for D, Hq, H, page, lens, new, window, (max_q, max_len), kernel, ranges in CASES:
        text = w4.kv4_attention_describe(len(lens), Hq, H, D, max_q, max_len, window, 0)
        say(text)
        split = "splits=1 " not in text
        if kernel:
            assert kernel in text, text
        if kernel and ranges:
            assert split, text
        seen.add((D, text.split(",")[1], split))
    for D in (64, 128, 256):
        assert (D, "128", True) in seen and {r for d, r, _ in seen if d == D} >= {"8", "16", "128"}


@pytest.mark.parametrize("queries,planned", [(1, 1), (5, 5), (40, 2048)])
@pytest.mark.parametrize("power", [9, 12, 30, 60])
def test_a_large_query_costs_its_neighbours_nothing(queries, planned, power):
    """Every third row 2^power as large as the others: those keep the bounds
    that follow from their own size."""
    import torch
    rng = np.random.default_rng(600 + power)
    page, H, Hq, D, n = 32, 1, 8, 128, 300
    pages = -(-n // page)
    table = np.arange(pages, dtype=np.int32)[None]
    max_len = 6000 if planned > queries else n
    say("attention neighbours", queries, power)
    k, v = rng.standard_normal((2, n, H, D)).astype(np.float32)
    cache = torch.empty((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
    K, V = (torch.from_numpy(x).half().cuda() for x in (k, v))
    w4.kv4_append(K, V, torch.arange(n, dtype=torch.int32, device="cuda"), cache)
    qs = rng.standard_normal((queries * Hq, D)).astype(np.float32)
    qs[::3] *= 2.0 ** power
    q = torch.from_numpy(qs.reshape(queries, Hq, D)).bfloat16().cuda()
    starts, i32 = np.array([0, queries]), dict(dtype=torch.int32, device="cuda")
    O, L = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    w4.kv4_attention(q, cache, torch.tensor(table, **i32), torch.tensor([n], **i32),
                     torch.tensor(starts, **i32), O, L, D ** -0.5, 0, planned, max_len,
                     w4.alloc_kv4_workspace(1, Hq, H, D, planned, max_len))
    torch.cuda.synchronize()
    want, lse, weight, size, floor, reach = _reference(q, cache, table, [n], starts, D ** -0.5, 0)
    small = np.arange(queries * Hq).reshape(queries, Hq) % 3 != 0
    bound = (2.0 ** -8 * np.abs(want) + 2.0 ** -25 * (1 + floor) + 2.0 ** -11 * weight
             + (16 * U * reach[..., None] + (64 + n / 32) * U) * size)
    err = np.abs(O.double().cpu().numpy() - want)
    assert np.isfinite(O.float().cpu().numpy()).all()
    assert (err <= bound)[small].all(), float((err / bound)[small].max())
    got = L.double().cpu().numpy()
    assert (np.abs(got - lse) <= 8 * U * reach + 64 * U * (1 + np.abs(lse)))[small].all()
