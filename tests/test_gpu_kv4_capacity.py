"""Scheduler steps with more new tokens than the token buffers hold: a request
whose tokens do not all fit is refused, so that no length ever covers a token
that was not stored.  Whole numbers are compared bit for bit."""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import kv4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

NAMES = ("lens_out", "table", "ring", "state_out", "q_start", "slots", "positions")


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,page,width,grow", [
    (1, 16, 4, 40), (3, 16, 4, 30), (200, 16, 9, 12), (257, 32, 9, 70), (1000, 16, 40, 100),
    (4096, 128, 5, 3)])
def test_tables_at_every_kind_of_capacity(B, page, width, grow, alias):
    import torch
    rng = np.random.default_rng(B + 9)
    lens = rng.integers(0, width * page + 1, B)
    kind = rng.random(B)
    want = np.where(kind < 0.7, lens + rng.integers(0, grow + 1, B),
                    np.where(kind < 0.8, np.maximum(0, lens - rng.integers(0, 3 * page, B)), lens))
    used = -(-lens // page)
    pages = int(used.sum()) + B * (grow // page + 2)
    ids, at = rng.permutation(pages), 0
    table = np.full((B, width), -1, np.int32)
    for b in range(B):
        table[b, : used[b]] = ids[at: at + used[b]]
        at += used[b]
    head = int(rng.integers(0, pages))
    ring = np.full(pages, -9, np.int32)
    ring[(head + np.arange(pages - at)) % pages] = ids[at:]
    total = int(np.maximum(0, want - lens).sum())
    ends = np.cumsum(np.maximum(0, want - lens))
    some = int(ends[B // 2])                       # a request's tokens end there
    for capacity in sorted({0, 1, some - 1, some, some + 1, total // 3, total - 1, total} - {-1}):
        for count in (pages - at, (pages - at) // 3):
            say("tables capacity", B, capacity, total, count, alias)
            state = [head, count, 0, 0]
            i32 = dict(dtype=torch.int32, device="cuda")
            d = [torch.tensor(x, **i32) for x in (lens, want, table, ring, state)]
            lens_out = d[0] if alias else torch.full((B,), -7, **i32)
            state_out = d[4] if alias else torch.zeros(4, **i32)
            rest = [torch.full((n,), -7, **i32) for n in (B + 1, capacity, capacity)]
            w4.kv4_tables(*d, lens_out, state_out, *rest, page)
            torch.cuda.synchronize()
            expect = ref.tables(lens, want, table, ring, state, capacity, page)
            got = (lens_out, d[2], d[3], state_out, *rest)
            for name, g, e in zip(NAMES, got, expect):
                assert np.array_equal(g.cpu().numpy(), e), name


@pytest.mark.parametrize("short", [0, 1, 8, 24])
def test_attention_after_a_step_that_did_not_fit_reads_stored_tokens_only(short):
    """tables -> append -> attention over a cache whose parameters are NaN: two
    prompts, the token buffers ``short`` too small, then a step for what is
    held.  No row of a served request is NaN, and the lengths say which are."""
    import torch
    say("capacity attention", short)
    B, page, width, H, Hq, D = 2, 16, 4, 1, 4, 64
    pages, total = 8, 64
    capacity = total - short
    cache = torch.full((pages, H, page, D + 8), 0xFF, dtype=torch.uint8, device="cuda")
    table, ring, state = w4.alloc_kv4_pages(pages, B, width)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, want = torch.zeros(B, **i32), torch.full((B,), 32, **i32)
    starts, slots, pos = (torch.full((n,), -7, **i32) for n in (B + 1, capacity, capacity))
    gen = torch.Generator(device="cuda").manual_seed(short)
    kv = torch.randn((2, capacity, H, D), device="cuda", generator=gen).half()
    Q = torch.randn((capacity, Hq, D), device="cuda", generator=gen).half()
    w4.kv4_tables(lens, want, table, ring, state, lens, state, starts, slots, pos, page)
    w4.kv4_append(kv[0], kv[1], slots, cache)
    O, L = torch.full_like(Q, 9.0), torch.full((capacity, Hq), 9.0, device="cuda")
    ws = w4.alloc_kv4_workspace(B, Hq, H, D, 32, 32)
    w4.kv4_attention(Q, cache, table, lens, starts, O, L, 0.125, 0, 32, 32, ws)
    torch.cuda.synchronize()
    served = 1 if short else 2
    assert lens.tolist() == [32] * served + [0] * (2 - served)
    assert int(state[2]) == 2 - served
    assert torch.isfinite(O[:32 * served].float()).all() and torch.isfinite(L[:32 * served]).all()
    # rows of the refused request see nothing, since it holds nothing
    assert bool((O[32 * served:] == 0).all()) and bool((L[32 * served:] == -float("inf")).all())
    # a decode step for both, over what they hold
    want.copy_(lens + 1)
    one = [torch.full((n,), -7, **i32) for n in (B + 1, B, B)]
    w4.kv4_tables(lens, want, table, ring, state, lens, state, *one, page)
    w4.kv4_append(kv[0, :B], kv[1, :B], one[1], cache)
    O, L = torch.full_like(Q[:B], 9.0), torch.full((B, Hq), 9.0, device="cuda")
    w4.kv4_attention(Q[:B], cache, table, lens, one[0], O, L, 0.125, 0, 1, 64,
                     w4.alloc_kv4_workspace(B, Hq, H, D, 1, 64))
    torch.cuda.synchronize()
    assert torch.isfinite(O.float()).all() and torch.isfinite(L).all()


def test_the_most_requests_of_a_call_under_a_graph():
    """4096 requests, whose sums take more shared memory than a launch gets
    unasked, replayed in place."""
    import torch
    say("tables graph 4096")
    B, page, width, capacity = w4.KV4_MAX_REQUESTS, 16, 4, 6000
    pages = B * width
    rng = np.random.default_rng(12)
    table, ring, state = w4.alloc_kv4_pages(pages, B, width)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, want = torch.zeros(B, **i32), torch.zeros(B, **i32)
    rest = [torch.zeros(n, **i32) for n in (B + 1, capacity, capacity)]
    held = [x.cpu().numpy() for x in (lens, table, ring, state)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.kv4_tables(lens, want, table, ring, state, lens, state, *rest, page)
    for i in range(6):
        w = np.clip(held[0] + rng.integers(-6, 4, B), 0, 64).astype(np.int32)
        want.copy_(torch.from_numpy(w))
        graph.replay()
        torch.cuda.synchronize()
        expect = ref.tables(held[0], w, *held[1:], capacity, page)
        for name, g, e in zip(NAMES, (lens, table, ring, state, *rest), expect):
            assert np.array_equal(g.cpu().numpy(), e), (i, name)
        held = expect[:4]
