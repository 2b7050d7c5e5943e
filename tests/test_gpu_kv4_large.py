"""kv4_attention where logits are so large that FP32 resolves them coarsely or
hardly holds them: every row that sees a key is an average of values, and the
keys that FP32 cannot tell from the largest are the only ones that may be in it.

Tolerances, derived from the arithmetic.  A logit is off by at most d = eight
roundings of the largest magnitude it is summed from (as in the other
attention tests), so a key may count as the largest if its exact logit is
within 2 d of it; keys 60 below those weigh less than n e^-60.  The output
lies between the smallest and the largest value of the keys that are left,
widened by its own rounding (eps/2), the weights' rounding to FP16 (2^-11 of
scale |code - 8|; FP16 calls carry the remainder: 2^-21), half of FP16's
smallest step at the largest weight for each of n keys, and FP32 sums of n
terms (64 + n/32 roundings).  lse is off by d and 64 roundings of 1 + |lse|.
"""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import kv4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
# queries of the request, planned: row tiles of 8, 16 and 128 (8 heads on one)
KERNELS = [(1, 1), (5, 5), (40, 2048)]


def _case(seed, n, queries, planned, power, every, dtype, zero=False, page=32, D=128, Hq=8):
    """One request of n tokens whose last ``queries`` are asked.  Rows
    ``::every`` are 2^power as large as the others: BF16 queries are, FP16
    calls get it by their scale (every row then).  Returns everything that
    ``_verify`` compares."""
    import torch
    rng = np.random.default_rng(seed)
    pages = -(-n // page)
    table = rng.permutation(pages).astype(np.int32)[None]
    k, v = rng.standard_normal((2, pages * page, 1, D)).astype(np.float32)
    cache = torch.empty((pages, 1, page, D + 8), dtype=torch.uint8, device="cuda")
    K, V = (torch.from_numpy(x).half().cuda() for x in (k, v))
    w4.kv4_append(K, V, torch.arange(pages * page, dtype=torch.int32, device="cuda"), cache)
    qs, scale = rng.standard_normal((queries * Hq, D)), D ** -0.5
    if dtype == "bfloat16":
        qs[::every] *= 2.0 ** power
    else:
        scale *= 2.0 ** power
    if zero:
        qs[1::3] = 0
    q = torch.from_numpy(qs.reshape(queries, Hq, D).astype(np.float32)).to(
        getattr(torch, dtype)).cuda()
    max_len = 6000 if planned > queries else n
    say("attention large", n, queries, power, every, dtype,
        w4.kv4_attention_describe(1, Hq, 1, D, planned, max_len))
    O = torch.full_like(q, 9.0)
    L = torch.full(q.shape[:2], 9.0, dtype=torch.float32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    w4.kv4_attention(q, cache, torch.tensor(table, **i32), torch.tensor([n], **i32),
                     torch.tensor([0, queries], **i32), O, L, scale, 0, planned, max_len,
                     w4.alloc_kv4_workspace(1, Hq, 1, D, planned, max_len))
    torch.cuda.synchronize()
    return q, cache, table, n, np.float32(scale).astype(np.float64), O, L


def _verify(case, decided):
    """Every row against the bounds above; at least ``decided`` of the rows
    have to have a single key that may be the largest."""
    import torch
    q, cache, table, n, scale, O, L = case
    page, T, Hq = cache.shape[2], q.shape[0], q.shape[1]
    eps = torch.finfo(q.dtype).eps / 2
    step = 2.0 ** -11 if q.dtype is torch.bfloat16 else 2.0 ** -21
    j = np.arange(n)
    slots = table[0, j // page].astype(np.int64) * page + j % page
    (kc, ks, kz), (vc, vs, vz) = ref.load(cache.cpu().numpy(), slots)
    key = kc[:, 0] * ks + kz
    value = vc[:, 0] * vs + vz
    rough = vs * np.abs(vc[:, 0])
    size = 15 * vs[:, 0] + np.abs(vz[:, 0])
    qd, o, lse = (x.double().cpu().numpy() for x in (q, O, L))
    alone = 0
    for t in range(T):
        m = n - T + t + 1
        reach = (23 * ks[:m, 0] + np.abs(kz[:m, 0])).max()
        for h in range(Hq):
            x = scale * (key[:m] @ qd[t, h])
            d = 8 * U * scale * np.abs(qd[t, h]).sum() * reach
            top = x.max()
            near = x >= top - 2 * d - 60
            alone += near.sum() == 1
            slack = (2.0 ** -25 * (1 + 8 * m * vs[:m].max()) + step * rough[:m][near].max(0)
                     + ((64 + m / 32) * U + m * np.exp(-60.0)) * size[:m].max())
            lo, hi = value[:m][near].min(0), value[:m][near].max(0)
            assert (o[t, h] >= lo - eps * np.abs(lo) - slack).all(), (t, h, top)
            assert (o[t, h] <= hi + eps * np.abs(hi) + slack).all(), (t, h, top)
            want = top + np.log(np.exp(x - top).sum())
            assert abs(lse[t, h] - want) <= d + 64 * U * (1 + abs(want)), (t, h, want)
    assert alone >= decided * T * Hq, alone


@pytest.mark.parametrize("queries,planned", KERNELS)
@pytest.mark.parametrize("dtype,every", [("bfloat16", 1), ("bfloat16", 3), ("float16", 1)])
@pytest.mark.parametrize("power", [12, 20, 26, 28, 30, 33, 40, 60, 90])
def test_large_logits_keep_their_largest_key(queries, planned, dtype, every, power):
    _verify(_case(700 + power, 300, queries, planned, power, every, dtype),
            0.9 if every == 1 else 0.3)


@pytest.mark.parametrize("queries,planned", KERNELS)
@pytest.mark.parametrize("power", [102, 106, 110])
def test_rows_whose_every_logit_is_far_below_zero_are_not_empty(queries, planned, power):
    """A prompt from its first token: the first rows see few keys, half of them
    with negative logits only, past any finite stand-in for "no key yet"."""
    for seed in range(3):
        _verify(_case(720 + power + 1000 * seed, queries, queries, planned, power, 1, "bfloat16"),
                0.5)


@pytest.mark.parametrize("queries,planned", KERNELS)
@pytest.mark.parametrize("every", [1, 3])
@pytest.mark.parametrize("power", [100, 115, 122, 125])
def test_queries_at_the_end_of_their_range(queries, planned, every, power):
    """BF16 queries up to their type's end, whose logits FP32 still holds, and
    rows of zeros beside them."""
    _verify(_case(760 + power, 300, queries, planned, power, every, "bfloat16", zero=True), 0.1)


@pytest.mark.parametrize("queries,planned", KERNELS)
@pytest.mark.parametrize("power", [100, 110, 120])
def test_scales_of_any_size(queries, planned, power):
    """The same by the scale of the call, with FP16 queries."""
    _verify(_case(780 + power, 300, queries, planned, power, 1, "float16", zero=True), 0.5)


@pytest.mark.parametrize("queries,planned", KERNELS)
def test_small_queries_under_a_large_scale(queries, planned):
    """Ordinary logits as 2^-95 times 2^95 are those of 1 times 1, bit for bit."""
    import torch
    results = []
    for power in (0, 95):
        rng = np.random.default_rng(790)
        n, page, Hq, D = 200, 32, 8, 128
        k, v = rng.standard_normal((2, 224, 1, D)).astype(np.float32)
        cache = torch.empty((7, 1, page, D + 8), dtype=torch.uint8, device="cuda")
        K, V = (torch.from_numpy(x).half().cuda() for x in (k, v))
        w4.kv4_append(K, V, torch.arange(224, dtype=torch.int32, device="cuda"), cache)
        q = torch.from_numpy(rng.standard_normal((queries, Hq, D)) * 2.0 ** -power).to(
            torch.float32).bfloat16().cuda()
        max_len = 6000 if planned > queries else n
        say("attention scale", queries, power)
        i32 = dict(dtype=torch.int32, device="cuda")
        O, L = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        w4.kv4_attention(q, cache, torch.arange(7, **i32)[None], torch.tensor([n], **i32),
                         torch.tensor([0, queries], **i32), O, L, D ** -0.5 * 2.0 ** power, 0,
                         planned, max_len, w4.alloc_kv4_workspace(1, Hq, 1, D, planned, max_len))
        torch.cuda.synchronize()
        results.append((O, L))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("queries,planned", KERNELS)
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("power", [30, 105, 124])
def test_large_rows_of_other_head_sizes(queries, planned, D, power):
    _verify(_case(800 + power, 200, queries, planned, power, 2, "bfloat16", zero=True, D=D), 0.2)


@pytest.mark.parametrize("queries,planned", KERNELS)
@pytest.mark.parametrize("power", [30, 124])
def test_large_rows_over_joined_ranges(queries, planned, power):
    """More tokens than a range holds: parts with unlike references are joined."""
    _verify(_case(820 + power, 1500, queries, planned, power, 2, "bfloat16", page=64), 0.4)
