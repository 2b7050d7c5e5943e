"""Queries, keys, values and outputs as parts of one buffer that lie between
each other, head by head: the bits of separate tensors."""

from __future__ import annotations

import pytest

import weight_only_int4_gemm_amd as w4
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,H,D,by_token", [(1, 4, 128, False), (37, 8, 64, False),
                                            (1100, 2, 128, False), (50, 3, 256, True)])
def test_a_layer_in_one_interleaved_buffer(dtype, T, H, D, by_token):
    import torch
    say("interleaved", dtype, T, H, D, by_token)
    gen = torch.Generator(device="cuda").manual_seed(T)
    shape = (H, T, 3, D) if by_token else (T, H, 3, D)
    one = torch.randn(shape, device="cuda", generator=gen).to(getattr(torch, dtype))
    if by_token:
        one = one.transpose(0, 1)
    q, k, v = one.unbind(2)
    apart = [x.contiguous() for x in (q, k, v)]
    page, i32 = 16, dict(dtype=torch.int32, device="cuda")
    pages = -(-T // page) + 1
    slots = torch.arange(T, **i32)
    pos = torch.arange(T, **i32)[None] * 3
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    table, lens = torch.arange(pages, **i32)[None], torch.tensor([T], **i32)
    starts = torch.tensor([0, T], **i32)
    ws = w4.alloc_kv4_workspace(1, H, H, D, T, T)
    results = []
    for x, y, z in ((q, k, v), apart):
        cache = torch.zeros((pages, H, page, D + 8), dtype=torch.uint8, device="cuda")
        keys = y.clone()
        w4.kv4_rope_append(x, y, z, x, pos, freq, (D // 2,), w4.KV4_ROPE_HALVES, slots, cache)
        assert torch.equal(y, keys)
        O = z if x is q else torch.zeros_like(x)     # the values are stored: their place is free
        w4.kv4_attention(x, cache, table, lens, starts, O, None, D ** -0.5, 0, T, T, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, keys)
        results.append((x.clone(), cache, O.clone()))
    for a, b in zip(*results):
        assert torch.equal(a, b)
