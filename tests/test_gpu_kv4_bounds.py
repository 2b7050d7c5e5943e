"""kv4_attention with every row held to bounds of its own size: queries of any
size beside each other, and sampled rows of a prompt as long as prompts are.

Tolerances as for the other attention tests: the output's rounding, the
rounding of each weight to FP16 (2^-11; FP16 calls carry the remainder:
2^-21), half of FP16's smallest step at the largest weight, eight roundings
of the largest magnitude in a score of the same row, and sums of n terms in
FP32 taken as 64 + n/32 roundings of the sum of magnitudes.
"""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import kv4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _verify(q, cache, table, lens, starts, scale, O, L, rows):
    """Rows (t, h) against 64 bits."""
    import torch
    page, Hq = cache.shape[2], q.shape[1]
    eps = torch.finfo(q.dtype).eps / 2
    step = 2.0 ** -11 if q.dtype is torch.bfloat16 else 2.0 ** -21
    host = cache.cpu().numpy()
    loaded = {}
    for t, h in rows:
        b = int(np.searchsorted(starts, t, side="right")) - 1
        n = lens[b] - (starts[b + 1] - starts[b]) + (t - starts[b]) + 1
        g = h // (Hq // cache.shape[1])
        if b not in loaded:
            j = np.arange(lens[b])
            loaded[b] = ref.load(host, table[b, j // page].astype(np.int64) * page + j % page)
        (kc, ks, kz), (vc, vs, vz) = ([x[:n, g] for x in part] for part in loaded[b])
        x = q[t, h].double().cpu().numpy()
        reach = scale * np.abs(x).sum() * (23 * ks + np.abs(kz)).max()
        s = scale * ((kc * ks[:, None] + kz[:, None]) @ x)
        p = np.exp(s - s.max())
        lse = s.max() + np.log(p.sum())
        p /= p.sum()
        want = p @ (vc * vs[:, None] + vz[:, None])
        bound = (eps * np.abs(want) + 2.0 ** -25 * (1 + 8 * n * (p * vs).max())
                 + step * ((p * vs) @ np.abs(vc))
                 + (16 * U * reach + (64 + n / 32) * U) * (p * (15 * vs + np.abs(vz))).sum())
        err = np.abs(O[t, h].double().cpu().numpy() - want)
        assert (err <= bound).all(), (t, h, float((err / bound).max()))
        assert abs(float(L[t, h]) - lse) <= 8 * U * reach + 64 * U * (1 + abs(lse)), (t, h)


@pytest.mark.parametrize("queries,planned", [(1, 1), (5, 5), (40, 2048)])
@pytest.mark.parametrize("powers", [(-120, -40, 3, 0, -7, -1, 2, -80), (0, -9, -11, -20, 4, 5, 6, 7),
                                    (-30, -31, -32, -90, -50, -60, -70, -33)])
def test_queries_of_any_size_within_their_own_bounds(queries, planned, powers):
    """A power of two per head, so that every tile holds them all."""
    import torch
    rng = np.random.default_rng(900 + queries)
    page, Hq, D, n = 16, 8, 128, 500
    pages = -(-n // page)
    table = np.arange(pages, dtype=np.int32)[None]
    k, v = rng.standard_normal((2, n, 1, D)).astype(np.float32)
    cache = torch.empty((pages, 1, page, D + 8), dtype=torch.uint8, device="cuda")
    K, V = (torch.from_numpy(x).half().cuda() for x in (k, v))
    w4.kv4_append(K, V, torch.arange(n, dtype=torch.int32, device="cuda"), cache)
    qs = rng.standard_normal((queries, Hq, D)) * np.exp2(np.array(powers, float))[None, :, None]
    q = torch.from_numpy(qs.astype(np.float32)).bfloat16().cuda()
    max_len = 6000 if planned > queries else n
    say("attention own bounds", queries, powers)
    i32 = dict(dtype=torch.int32, device="cuda")
    O, L = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    w4.kv4_attention(q, cache, torch.tensor(table, **i32), torch.tensor([n], **i32),
                     torch.tensor([0, queries], **i32), O, L, 0.5, 0, planned, max_len,
                     w4.alloc_kv4_workspace(1, Hq, 1, D, planned, max_len))
    torch.cuda.synchronize()
    _verify(q, cache, table, [n], [0, queries], 0.5, O, L,
            [(t, h) for t in range(queries) for h in range(Hq)])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("Hq,H", [(16, 2), (64, 8)])
def test_sampled_rows_of_long_prompts(dtype, Hq, H):
    """Two chunks of 2048 and 1500 queries over 6000 and 1500 tokens: tiles of
    16 rows with few heads, full ones of 128 with many."""
    import torch
    rng = np.random.default_rng(910)
    page, D = 64, 128
    lens, new = [6000, 1500], [2048, 1500]
    text = w4.kv4_attention_describe(2, Hq, H, D, 2048, 6000)
    say("attention long prompts", dtype, text)
    assert ("rows" if Hq == 64 else "tokens") in text
    used = [-(-n // page) for n in lens]
    pages = sum(used)
    ids = rng.permutation(pages)
    table = np.full((2, max(used)), -1, np.int32)
    table[0, :used[0]], table[1, :used[1]] = ids[:used[0]], ids[used[0]:]
    k, v = rng.standard_normal((2, pages * page, H, D)).astype(np.float32)
    cache = torch.empty((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
    K, V = (torch.from_numpy(x).half().cuda() for x in (k, v))
    w4.kv4_append(K, V, torch.arange(pages * page, dtype=torch.int32, device="cuda"), cache)
    starts = [0, 2048, 3548]
    q = torch.from_numpy(rng.standard_normal((3548, Hq, D)).astype(np.float32) * 1.3).to(
        getattr(torch, dtype)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    O, L = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    w4.kv4_attention(q, cache, torch.tensor(table, **i32), torch.tensor(lens, **i32),
                     torch.tensor(starts, **i32), O, L, D ** -0.5, 0, 2048, 6000,
                     w4.alloc_kv4_workspace(2, Hq, H, D, 2048, 6000))
    torch.cuda.synchronize()
    assert torch.isfinite(O.float()).all() and torch.isfinite(L).all()
    rows = [(t, int(rng.integers(Hq))) for t in (0, 1, 15, 16, 127, 2047, 2048, 2049, 3547)]
    rows += [(int(rng.integers(3548)), int(rng.integers(Hq))) for _ in range(40)]
    _verify(q, cache, table, lens, starts, D ** -0.5, O, L, rows)
