"""moe_route where its forms and lanes change: sigmoid scores far below what
FP32 holds, and every compiled number of lanes, experts and group marks.

Tolerances of the weights, from the arithmetic (U = 2^-24, an FP32 rounding):
* sigmoid: scores and their sum are 64-bit numbers, whose roundings are far
  below U; the quotient is rounded to FP32 once and times the scale once:
  2 U, taken as 3 U for the second order and the 64-bit part.  So it is with a
  bias or marks of two, whatever the score.
* softmax otherwise: the exponent's difference d is rounded once (|d| U) and
  the exponential is good to 2 U; sums of at most 32 or 1024 such terms in 64
  partial ones, and two divisions: (2 max|d| + 64) U.
Below 2^-126 a rounding is half of FP32's smallest step, 2^-149: the quotient's
times the scale, and the product's, (scale + 1) / 2 steps; taken as one more,
for an exponential in 32 bits.
"""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import moe_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = 2.0 ** -149


def _check(rows, T, name, bias, k, softmax, **kind):
    """``rows`` distinct tokens, repeated to T: every place of a workgroup gets
    every one of them in turn."""
    import torch
    n, E = rows.shape
    x = torch.from_numpy(np.asarray(rows, np.float32)).to(getattr(torch, name)).cuda()
    exact = x.double().cpu().numpy()
    x = x[torch.arange(T, device="cuda") % n].contiguous()
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    w4.moe_route(x, b, ids, w, score=w4.MOE_SOFTMAX if softmax else w4.MOE_SIGMOID, **kind)
    want_ids, want_w = (v[np.arange(T) % n]
                        for v in ref.route(exact, bias, k, softmax=softmax, **kind))
    got_ids, got_w = ids.cpu().numpy(), w.double().cpu().numpy()
    assert np.array_equal(got_ids, want_ids), np.argwhere(got_ids != want_ids)[:4]
    by_logit = bias is None and (kind.get("groups", 1) == 1 or kind.get("group_best", 1) == 1)
    relative = 3 * U
    if softmax and by_logit:
        relative = (2 * float(exact.max() - exact.min()) + 64) * U
    least = ((kind.get("scale", 1.0) + 1) / 2 + 1) * STEP
    bad = ~(np.abs(got_w - want_w) <= relative * np.abs(want_w) + least)
    assert not bad.any(), (int(bad.sum()), got_w[bad][:4], want_w[bad][:4])


@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("T", [7, 4103])                     # 64 and 16 lanes a token
@pytest.mark.parametrize("E,groups", [(8, 1), (96, 1), (96, 6), (256, 8), (640, 1)])
def test_sigmoid_of_very_negative_logits(E, groups, T, name):
    say("sigmoid", E, groups, T, name)
    rng = np.random.default_rng(E)
    rows = np.stack([
        np.full(E, -95.0), -95.0 - np.arange(E) % 3,           # below 2^-126, tied or not
        -rng.uniform(80, 300, E), -rng.uniform(86, 105, E),
        np.where(np.arange(E) == E - 2, -80.0, -90.0),         # one FP32 would hold, others not
        np.where(np.arange(E) % 5 == 0, 3.0, -200.0),
        np.full(E, -700.0) + rng.integers(0, 4, E),
        np.where(np.arange(E) < 3, -100.0, -np.inf),           # fewer than k
        np.full(E, -2000.0 if name != "float16" else -1500.0)])  # 0 in 64 bits too
    k = min(6, E)
    for renorm in (True, False):
        for scale in (1.0, 2.5):
            for bias in (None, np.zeros(E)):
                _check(rows, T, name, bias, k, False, groups=groups,
                       top_groups=max(1, groups // 2), renorm=renorm, scale=scale)


# Experts, choices, groups and groups kept.  From 4096 tokens on 16 lanes take a token (up to
# 16 experts always), with 1, 4, 8 or 16 experts a lane; a lane has two choices
# for k > 16 and up to four marks for more than 16 groups.
WIDE = [(16, 16, 1, 1), (17, 4, 1, 1), (60, 6, 1, 1), (60, 32, 4, 3), (64, 8, 8, 4), (64, 20, 32, 20),
        (64, 9, 64, 11), (128, 8, 1, 1), (128, 32, 32, 12), (128, 12, 64, 30), (160, 6, 1, 1),
        (160, 32, 32, 15), (256, 8, 8, 4), (256, 32, 1, 1), (256, 32, 64, 33), (129, 17, 1, 1),
        (384, 32, 48, 17), (1000, 20, 40, 21)]


@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("T", [53, 4109])
@pytest.mark.parametrize("E,k,groups,top", WIDE)
def test_every_division_of_experts_among_lanes(E, k, groups, top, T, name):
    say("route lanes", E, k, groups, top, T, name)
    rng = np.random.default_rng(E * 64 + groups)
    rows = rng.standard_normal((53, E)) * 2.0
    rows[1], rows[2, ::2], rows[3, 1::2] = 0.5, -np.inf, np.nan
    rows[4] = np.repeat(rng.standard_normal(-(-E // 4)), 4)[:E]  # ties of four
    rows[5, :E - 1] = -np.inf
    bias = np.round(rng.standard_normal(E) * 0.2, 2).astype(np.float32).astype(np.float64)
    kind = dict(groups=groups, top_groups=top)
    for softmax in (True, False):
        finite = np.where(np.isfinite(rows), rows, 0.25) if softmax else rows
        _check(finite, T, name, None, k, softmax, **kind)
        _check(rows, T, name, bias, k, softmax, group_best=2, renorm=False, scale=2.5, **kind)
        _check(rows, T, name, bias, k, softmax, group_best=1, **kind)
        if groups > 1:
            _check(rows, T, name, None, k, softmax, group_best=2, **kind)
