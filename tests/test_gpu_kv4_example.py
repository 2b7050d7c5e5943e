"""The example layer: prompt and decode steps, launched one by one and from a
graph, and its attention against the reference over the cache it filled."""

from __future__ import annotations

import numpy as np
import pytest

import weight_only_int4_gemm_amd as w4
from oracle import kv4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


def _layer(requests, max_len):
    from examples import kv4_decode as ex
    return ex, ex.Layer(512, 4, 2, 64, requests, max_len, page=16)


@pytest.mark.parametrize("requests,prompt,steps", [(1, 1, 3), (3, 37, 5)])
def test_steps_from_a_graph_equal_steps_launched_one_by_one(requests, prompt, steps):
    import torch
    say("example", requests, prompt, steps)
    results = []
    for graph in (False, True):
        ex, layer = _layer(requests, prompt + steps)
        y, last, _ = ex.run(layer, prompt, steps, graph=graph)
        assert layer.lens.tolist() == [prompt + steps] * requests
        assert int(layer.state[2]) == 0
        assert torch.isfinite(last.float()).all() and float(last.float().abs().max()) > 0
        results.append((y, last, layer.table))
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_attention_of_the_layer_matches_the_reference():
    """The queries the layer rotated in place and the cache it filled, through
    the reference: FP16 rounding of the output, the remainder of the weights'
    rounding (2^-21), FP16's smallest step at the largest weight, and sums in
    FP32."""
    import torch
    say("example attention")
    requests, prompt = 2, 45
    ex, layer = _layer(requests, prompt)
    b = layer.buffers(requests * prompt, prompt)
    b["x"].normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    b["want"].fill_(prompt)
    layer.forward(b)
    torch.cuda.synchronize()
    q = b["qkv"][:, :4].double().cpu().numpy()
    want, lse, weight, size, floor, reach = ref.attention(
        q, layer.cache.cpu().numpy(), layer.table.cpu().numpy(), layer.lens.cpu().numpy(),
        layer.starts.cpu().numpy(), 64 ** -0.5)
    assert np.isfinite(lse).all()
    u = 2.0 ** -24
    bound = (2.0 ** -11 * np.abs(want) + 2.0 ** -25 * (1 + floor) + 2.0 ** -21 * weight
             + (16 * u * reach[..., None] + (64 + prompt / 32) * u) * size)
    got = b["attn"].double().cpu().numpy()
    assert (np.abs(got - want) <= bound).all()
    # and the product after it sees that output
    W = torch.empty((256, 512), dtype=torch.float16, device="cuda")
    w4.w4a16_dequant_debug(layer.out.packed, layer.out.scales, W, 256, 512, ex.GROUP)
    y = got.reshape(-1, 256) @ W.double().cpu().numpy()
    mag = np.abs(got.reshape(-1, 256)) @ np.abs(W.double().cpu().numpy())
    err = np.abs(b["y"].double().cpu().numpy() - y)
    assert (err <= 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + (256 + 64) * u * mag + 2.0 ** -10 * mag).all()
