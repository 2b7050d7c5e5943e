"""Sizes that no launch takes are refused as sizes: a grid has fewer than 2^32
threads, so at most 2^24 - 1 workgroups of 256."""

from __future__ import annotations

import re

import pytest

import weight_only_int4_gemm_amd as w4
from tests.test_kv4_abi import APPEND, DEVICE, FUSED, ROPE, SHAPE

GROUPS = (1 << 24) - 1


@pytest.fixture(scope="module")
def accepted():
    """What a call with fake addresses comes to once its sizes are accepted."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: without a device only")
    return DEVICE


@pytest.mark.parametrize("fn,base", [("kv4_rope", ROPE), ("kv4_append", APPEND),
                                     ("kv4_rope_append", FUSED)])
def test_tokens_of_a_call(fn, base, accepted):
    call = getattr(w4.load(), fn)
    # rows far enough apart in the address space for any T
    strides = {k: 256 for k in base if k.endswith("_token")}
    strides |= {k: 128 for k in base if k.endswith("_head")}
    heads = {k: 1 for k in ("H", "Hq") if k in base}
    at = 1 << 44
    fake = {}
    for k, v in base.items():
        if k in ("X", "Y", "Q", "K", "V", "Qout", "cache", "positions", "inv_freq", "slots"):
            fake[k], at = at, at + (1 << 40)
    args = {**base, **strides, **heads, **fake}
    for T, want in ((4 * GROUPS, accepted), (4 * GROUPS + 1, SHAPE), (1 << 30, SHAPE)):
        assert call(*{**args, "T": T}.values()) == want, T


@pytest.mark.parametrize("sizes", [
    # B, Hq, H, D, max_q, max_len
    (4096, 32, 32, 128, 16384, 16384),      # tiles of 128 rows
    (1 << 19, 32, 32, 128, 1, 1024),        # a token each
    (1 << 19, 32, 32, 128, 20, 1024),       # tiles of 16
])
def test_workgroups_of_an_attention_call(sizes):
    B, Hq, H, D, max_q, max_len = sizes

    def grid(B):
        return int(re.search(r"grid=(\d+)", w4.kv4_attention_describe(
            B, Hq, H, D, max_q, max_len, 0, 256)).group(1))
    with pytest.raises(w4.W4A16Error) as e:
        grid(B)
    assert e.value.name == "W4A16_ERR_SHAPE"
    lo, hi = 1, B                                   # the most requests that are accepted
    while hi - lo > 1:
        mid = (lo + hi) // 2
        try:
            grid(mid)
            lo = mid
        except w4.W4A16Error:
            hi = mid
    assert grid(lo) <= GROUPS < grid(lo) + grid(1) * 64 and lo >= B // 4


def test_no_plan_passes_the_limit():
    for B in (1, 64, 5000, 1 << 17, 1 << 20, 1 << 24):
        for Hq, H in ((1, 1), (64, 8), (1024, 1024)):
            for q in (1, 8, 100, 1 << 14, 1 << 20):
                for n in (1, 100000, 1 << 30):
                    try:
                        d = w4.kv4_attention_describe(B, Hq, H, 64, q, n, 0, 256)
                    except w4.W4A16Error:
                        continue
                    assert int(re.search(r"grid=(\d+)", d).group(1)) <= GROUPS


@pytest.mark.gpu
def test_rotation_of_the_most_tokens_a_call_takes():
    """8 GiB in place: the first and last rows, and some at 32-bit offsets'
    ends, are those of small calls."""
    import torch
    from tests.gpu_util import say
    T, D = 4 * GROUPS, 64
    say("rope", T)
    X = torch.empty((T, 1, D), dtype=torch.float16, device="cuda")
    X.view(-1)[: 1 << 20].normal_()
    step = 1 << 20
    for at in range(step, X.numel(), step):         # one pattern, everywhere
        n = min(step, X.numel() - at)
        X.view(-1)[at: at + n] = X.view(-1)[:n]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    freq = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    picks = [0, 5, (1 << 25) - 3, 1 << 25, (1 << 26) - 20, T - 9]
    small = []
    for t in picks:
        x = X[t: t + 9].clone()
        w4.kv4_rope(x, x, pos[:, t: t + 9].contiguous(), freq, (32,))
        small.append(x)
    w4.kv4_rope(X, X, pos, freq, (32,))
    torch.cuda.synchronize()
    for t, x in zip(picks, small):
        assert torch.equal(X[t: t + 9], x), t


@pytest.mark.gpu
def test_attention_of_the_most_workgroups_a_call_takes():
    import torch
    from tests.gpu_util import say
    B, H, D, page = 16383, 1024, 64, 16
    text = w4.kv4_attention_describe(B, H, H, D, 1, 16)
    say("attention", text)
    assert int(re.search(r"grid=(\d+)", text).group(1)) == B * H
    cache = w4.alloc_kv4_cache(1, H, D, page)
    kv = torch.randn((2, 1, H, D), device="cuda").half()
    i32 = dict(dtype=torch.int32, device="cuda")
    w4.kv4_append(kv[0], kv[1], torch.zeros(1, **i32), cache)
    K, V = torch.empty((2, 1, H, D), dtype=torch.float16, device="cuda")
    w4.kv4_dequant_debug(torch.zeros(1, **i32), cache, K, V)
    Q = torch.ones((B, H, D), dtype=torch.float16, device="cuda")
    O = torch.full_like(Q, 9.0)
    w4.kv4_attention(Q, cache, torch.zeros((B, 1), **i32), torch.ones(B, **i32), None, O, None,
                     0.125, 0, 1, 16, w4.alloc_kv4_workspace(B, H, H, D, 1, 16))
    torch.cuda.synchronize()
    # one key: its values, to the last place of the sum and of the weight
    assert float((O[0].float() - V[0].float()).abs().max()) <= 2.0 ** -9 * float(V.abs().max())
    assert bool((O == O[0]).all())
