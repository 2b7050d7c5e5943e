"""An attention layer with 4-bit weights and a 4-bit key/value cache: a
prompt, then decode steps, each one graph launch.

    python examples/kv4_decode.py [--requests 64] [--prompt 2000] [--steps 50]

The default sizes are those of a Llama-2-7B layer (hidden 4096, 32 heads of
128 channels); weights and hidden states are random.  A step is

    w4a16_gemm        hidden states -> queries, keys, values
    kv4_tables        lengths -> page table, slots, positions
    kv4_rope_append   rotates queries and keys, stores keys and values
    kv4_attention     over the cache
    w4a16_gemm        attention output -> hidden states

and nothing in it returns to the host: lengths grow on the device.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import weight_only_int4_gemm_amd as w4
from synth import make_inputs

GROUP = 128


class Linear:
    """A weight in 4 bits, laid out once."""

    def __init__(self, K, N, seed):
        _, words, scales = make_inputs(1, K, N, GROUP, seed)
        self.K, self.N = K, N
        self.packed = w4.alloc_packed(K, N)
        w4.w4a16_repack(torch.from_numpy(words.view(np.int32)).cuda(), self.packed, K, N)
        # scaled so that a product has about the size of its input
        self.scales = torch.from_numpy(scales / np.float16(0.06 * K ** 0.5)).cuda()

    def __call__(self, x, out, workspace):
        w4.w4a16_gemm(x, self.packed, self.scales, out, x.shape[0], self.K, self.N, GROUP,
                      workspace)


class Layer:
    """One attention layer and the cache of ``requests`` requests of up to
    ``max_len`` tokens."""

    def __init__(self, hidden, heads, kv_heads, head_dim, requests, max_len, page=64,
                 max_tokens=None, seed=0):
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.page, self.max_len = page, max_len
        self.qkv = Linear(hidden, (heads + 2 * kv_heads) * head_dim, seed)
        self.out = Linear(heads * head_dim, hidden, seed + 1)
        width = -(-max_len // page)
        pages = requests * width
        self.cache = w4.alloc_kv4_cache(pages, kv_heads, head_dim, page)
        self.table, self.ring, self.state = w4.alloc_kv4_pages(pages, requests, width)
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.starts = torch.zeros(requests + 1, dtype=torch.int32, device="cuda")
        self.freq = 10000.0 ** (-torch.arange(head_dim // 2, dtype=torch.float64, device="cuda")
                                / (head_dim // 2))

    def buffers(self, tokens, max_q):
        """What a call of ``tokens`` tokens, at most ``max_q`` of a request, writes."""
        H, K, D = self.heads, self.kv_heads, self.head_dim
        f16 = dict(dtype=torch.float16, device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        requests = self.lens.numel()
        need = max(w4.w4a16_workspace_bytes(tokens, self.qkv.K, self.qkv.N, GROUP),
                   w4.w4a16_workspace_bytes(tokens, self.out.K, self.out.N, GROUP),
                   w4.kv4_attention_workspace_bytes(requests, H, K, D, max_q, self.max_len))
        return dict(max_q=max_q,
                    x=torch.zeros((tokens, self.qkv.K), **f16),
                    want=torch.zeros(requests, **i32),
                    qkv=torch.zeros((tokens, H + 2 * K, D), **f16),
                    attn=torch.zeros((tokens, H, D), **f16),
                    y=torch.zeros((tokens, self.out.N), **f16),
                    slots=torch.zeros(tokens, **i32), positions=torch.zeros(tokens, **i32),
                    workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))

    def forward(self, b):
        """b["x"] -> b["y"]; requests grow to b["want"] tokens."""
        H, K, D = self.heads, self.kv_heads, self.head_dim
        self.qkv(b["x"], b["qkv"].view(-1, self.qkv.N), b["workspace"])
        w4.kv4_tables(self.lens, b["want"], self.table, self.ring, self.state, self.lens,
                      self.state, self.starts, b["slots"], b["positions"], self.page)
        q, k, v = b["qkv"].split((H, K, K), dim=1)
        w4.kv4_rope_append(q, k, v, q, b["positions"], self.freq, (D // 2,),
                           w4.KV4_ROPE_HALVES, b["slots"], self.cache)
        w4.kv4_attention(q, self.cache, self.table, self.lens, self.starts, b["attn"], None,
                         D ** -0.5, 0, b["max_q"], self.max_len, b["workspace"])
        self.out(b["attn"].view(-1, H * D), b["y"], b["workspace"])
        return b["y"]


def run(layer, prompt, steps, graph=True, seed=0):
    """A prompt of ``prompt`` tokens per request, then ``steps`` tokens each,
    all of random hidden states.  Returns (the prompt's outputs, the last
    step's outputs, seconds of a step)."""
    requests = layer.lens.numel()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    first = layer.buffers(requests * prompt, prompt)
    first["x"].normal_(generator=gen)
    first["want"].fill_(prompt)
    y = layer.forward(first).clone()

    b = layer.buffers(requests, 1)
    inputs = torch.empty((steps, *b["x"].shape), dtype=torch.float16, device="cuda")
    inputs.normal_(generator=gen)

    def step():
        b["want"].copy_(layer.lens)
        b["want"].add_(1)
        layer.forward(b)

    launch = step
    if graph and steps:
        captured = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(captured):
            step()
        launch = captured.replay
    torch.cuda.synchronize()
    start = time.perf_counter()
    for i in range(steps):
        b["x"].copy_(inputs[i])
        launch()
    torch.cuda.synchronize()
    return y, b["y"], (time.perf_counter() - start) / max(1, steps)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=32)
    p.add_argument("--head-dim", type=int, default=128)
    p.add_argument("--requests", type=int, default=64)
    p.add_argument("--prompt", type=int, default=2000)
    p.add_argument("--steps", type=int, default=50)
    p.add_argument("--eager", action="store_true", help="launch kernels one by one")
    a = p.parse_args()
    layer = Layer(a.hidden, a.heads, a.kv_heads, a.head_dim, a.requests, a.prompt + a.steps)
    _, y, seconds = run(layer, a.prompt, a.steps, graph=not a.eager)
    size = w4.kv4_cache_bytes(*layer.cache.shape[:2], a.head_dim, layer.page)
    print(f"{a.requests} requests of {int(layer.lens[0])} tokens, cache {size / 2**20:.0f} MiB "
          f"({size / (2 * 2 * layer.cache.shape[0] * layer.page * a.kv_heads * a.head_dim):.2f} "
          f"of FP16): {seconds * 1e6:.1f} us per layer and step, "
          f"largest output {float(y.abs().max()):.3g}")


if __name__ == "__main__":
    main()
