"""moe_tables with room around its tensors: numbers of choices whose last chunk
is short, with many experts, where the chunks' counts need the most room."""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

GUARD = 4096                 # entries before, between and behind the tensors
MARK = -77


def _tables(ids, E):
    """By a stable sort (oracle/moe_ref.py loops over experts)."""
    flat = ids.reshape(-1).astype(np.int64)
    flat = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(flat, kind="stable").astype(np.int32)
    starts = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])])
    kept = int(starts[E])
    where = np.full(flat.size, -1, np.int32)
    where[order[:kept]] = np.arange(kept)
    order[kept:] = -1
    return starts.astype(np.int32), order, where


@pytest.mark.parametrize("T,k", [(16384, 1), (3277, 5), (2080, 8), (9000, 4), (87381, 3),
                                 (131072, 1)])
@pytest.mark.parametrize("E", [1, 7, 963, 964, 1000, 1024])
def test_tables_keep_to_their_tensors(T, k, E):
    import torch
    n = T * k
    say("tables bounds", T, k, E)
    rng = np.random.default_rng(n + E)
    for adjacent in (False, True):       # where right behind order, as an allocator may place it
        for most in (E, E + 40):
            ids = rng.integers(0 if most == E else -40, most, (T, k)).astype(np.int32)
            gap = 0 if adjacent else GUARD
            room = torch.full((3 * GUARD + gap + E + 1 + 2 * n,), MARK, dtype=torch.int32,
                              device="cuda")
            at, parts = GUARD, {}
            for name, size, after in (("starts", E + 1, GUARD), ("order", n, gap),
                                      ("where", n, GUARD)):
                parts[name] = (at, at + size)
                at += size + after
            view = {name: room[lo:hi] for name, (lo, hi) in parts.items()}
            w4.moe_tables(torch.from_numpy(ids).cuda(), view["starts"], view["order"],
                          view["where"].view(T, k))
            got = room.cpu().numpy()
            for name, want in zip(("starts", "order", "where"), _tables(ids, E)):
                lo, hi = parts[name]
                assert np.array_equal(got[lo:hi], want), (name, adjacent, most)
                got[lo:hi] = MARK
            assert (got == MARK).all(), (adjacent, most, np.flatnonzero(got != MARK)[:8])
