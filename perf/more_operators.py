"""Cases for the operators of expert layers and of layers in 8-bit floating point.

    route      router logits -> experts, weights and rows sorted by expert
                                                          (moe_route, moe_tables)
    quantize   16-bit rows -> e4m3 codes with a scale per 128 (w8a8_quantize)
    dense      product of e4m3 matrices with block scales     (w8a8_gemm)
    experts    a product with each row's own expert, in 4 or 8 bits:
               up    rows gathered from the tokens, SiLU of the gate half times
                     the up half                 (w4a16_moe_gemm, w8a8_moe_gemm)
               down  and the weighted sum over a token's experts  (moe_combine)

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits (routing scores in 64: experts next to the border of the
best k); with ``own`` true it calls the library.

Weights are held as the library's permuted layouts:

    w4a16  int32 [E][N/16][K/128][64 lanes][4 words]: lane l of word w holds
           codes k = 32 w + 8 (l / 16) + i, i = 0..7, of column l % 16, code i
           at nibble (0, 4, 1, 5, 2, 6, 3, 7)[i];  value (q - 8) * scale
    w8a8   e4m3 [E][N/16][K/128][2 halves][64 lanes][16]: lane l of half h
           holds k = 64 h + 16 (l / 16) + i of column l % 16
"""

import math
import random

import torch

own = False

_DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_NIBBLE = (0, 4, 1, 5, 2, 6, 3, 7)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a model with many experts in groups, scores by
        # sigmoid with a bias for balance
        dict(name="route decode 48", op="route", T=48, E=256, k=8, score="sigmoid", bias=1,
             groups=8, top_groups=4, group_best=2, renorm=1, scale=2.5, dtype="float32"),
        # a scheduler step full of prompts, softmax over all experts
        dict(name="route prefill 16384", op="route", T=16384, E=128, k=8, score="softmax", bias=0,
             groups=1, top_groups=1, group_best=1, renorm=1, scale=1.0, dtype="bfloat16"),
        # few large experts, an odd number of tokens
        dict(name="route few 4099", op="route", T=4099, E=8, k=2, score="softmax", bias=0,
             groups=1, top_groups=1, group_best=1, renorm=1, scale=1.0, dtype="float16"),
        # activations of a decode step before an 8-bit product: latency alone
        dict(name="quantize decode 32", op="quantize", T=32, K=4096, dtype="float16"),
        # and of a batch of prompts: bandwidth alone
        dict(name="quantize prefill 8192", op="quantize", T=8192, K=8192, dtype="bfloat16"),
        # one token through a square layer: the smallest call
        dict(name="dense one 4096x4096", op="dense", M=1, K=4096, N=4096, dtype="float16"),
        # a decode batch, odd, through a deep and narrow layer: few tiles, a long axis
        dict(name="dense batch 100 11008x4096", op="dense", M=100, K=11008, N=4096,
             dtype="bfloat16"),
        # prompts through a wide layer: matrix bound
        dict(name="dense prefill 4096 8192x28672", op="dense", M=4096, K=8192, N=28672,
             dtype="bfloat16"),
        # a decode step of many small experts: most are read for one or two rows
        dict(name="experts w8a8 up decode 24", op="experts", form="w8a8", part="up", T=24, E=128,
             k=8, K=2048, N=768, group=128, elsewhere=0, dtype="bfloat16"),
        # prompts through many small experts, loads unlike each other
        dict(name="experts w8a8 down prefill 8192", op="experts", form="w8a8", part="down", T=8192,
             E=64, k=6, K=1408, N=2048, group=128, elsewhere=0, dtype="bfloat16"),
        # a decode step of few large experts with 4-bit weights: cache-cold weight bandwidth
        dict(name="experts w4a16 down decode 9", op="experts", form="w4a16", part="down", T=9, E=8,
             k=2, K=11008, N=4096, group=128, elsewhere=0, dtype="float16"),
        # prompts through few large experts with 4-bit weights: matrix bound
        dict(name="experts w4a16 up prefill 4096", op="experts", form="w4a16", part="up", T=4096,
             E=8, k=2, K=4096, N=11008, group=128, elsewhere=0, dtype="float16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 100)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        case = _draw_one(rng)
        if _cost(case) <= most and _plain_bytes(case) <= 24e9:
            return case


def _plain_bytes(case):
    """About what the plain products hold at once, were the fullest expert to
    hold four times the mean."""
    if case["op"] == "dense":
        return 6 * case["K"] * case["N"]
    if case["op"] != "experts":
        return 0
    E, K, W = case["E"], case["K"], _columns(case)
    full = 4 * case["T"] * case["k"] + 16 * E
    return 8 * E * K * W + 4 * full * (K + 2 * W)


def _draw_one(rng):
    op = rng.choice(("route", "quantize", "dense", "dense", "experts", "experts", "experts"))
    dtype = rng.choice(("float16", "bfloat16"))
    if op == "route":
        E = rng.choice((4, 8, 16, 60, 64, 128, 160, 256, 384))
        groups = rng.choice((1, 1, 4, 8)) if E in (64, 128, 160, 256, 384) else 1
        top = rng.choice((groups // 4, groups // 2)) if groups > 1 else 1
        k = rng.choice([k for k in (1, 2, 4, 6, 8, 16) if k <= E * top // groups])
        bias = rng.randrange(2)
        return dict(op=op, T=_spread(rng, 1, 16384), E=E, k=k,
                    score=rng.choice(("softmax", "sigmoid")), bias=bias, groups=groups,
                    top_groups=top, group_best=rng.choice((1, 2)), renorm=rng.randrange(2),
                    scale=rng.choice((1.0, 2.5)), dtype=rng.choice(tuple(_DTYPES)))
    if op == "quantize":
        return dict(op=op, T=_spread(rng, 1, 16384), K=128 * _spread(rng, 1, 128), dtype=dtype)
    if op == "dense":
        return dict(op=op, M=_spread(rng, 1, 8192), K=128 * _spread(rng, 2, 144),
                    N=16 * _spread(rng, 8, 1800), dtype=dtype)
    K = 128 * _spread(rng, 2, 112)
    return dict(op=op, form=rng.choice(("w4a16", "w8a8")), part=rng.choice(("up", "down")),
                T=_spread(rng, 1, 8192), E=rng.choice((4, 8, 16, 60, 64, 128, 256)),
                k=rng.choice((1, 2, 4)) if rng.randrange(2) else rng.choice((2, 3, 4)), K=K,
                N=32 * _spread(rng, 4, 448), group=K if rng.randrange(4) == 0 else 128,
                elsewhere=int(rng.randrange(4) == 0), dtype=dtype)


def _columns(case):
    """Columns of an expert's weights."""
    return case["N"] * (2 if case["part"] == "up" else 1)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        # ids and weights out; ids in again, their order and its inverse out
        return {"bytes": T * E * size + T * k * (8 + 4 + 8) + 4 * E * (1 + case["bias"]),
                "flops": 6 * T * E}
    if op == "quantize":
        n = case["T"] * case["K"]
        return {"bytes": 3 * n + n // 32, "flops": 3 * n}
    if op == "dense":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": K * N + M * K + (M + -(-N // 128)) * K // 32 + 2 * M * N,
                "flops": 2 * M * K * N}
    T, E, k, K, N, W = (case["T"], case["E"], case["k"], case["K"], case["N"], _columns(case))
    all_experts = E * (2 if case["elsewhere"] else 1)
    rows = T * k * E / all_experts
    used = E * (1 - (1 - k / all_experts) ** T)      # experts that have a row
    if case["form"] == "w4a16":
        weights, row = K * W / 2 + 2 * (K // case["group"]) * W, 2 * K
    else:
        weights, row = K * W + 4 * (K // 128) * -(-W // 128), K + K // 32
    read = min(rows, T) if case["part"] == "up" else rows
    wrote = rows if case["part"] == "up" else T
    return {"bytes": int(used * weights + read * row + 2 * wrote * N + 8 * T * k),
            "flops": int(2 * rows * K * W)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    return _PREPARE[case["op"]](case, g)


def _randn(shape, g, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def _rand(shape, g):
    return torch.rand(shape, device="cuda", generator=g)


def _ints(shape):
    return torch.zeros(shape, device="cuda", dtype=torch.int32)


def _prepare_route(case, g):
    T, E, k = case["T"], case["E"], case["k"]
    # experts unlike each other in how often they are asked for
    logits = _randn((T, E), g) * 1.5 + _randn((1, E), g, scale=0.5)
    return dict(case=case, logits=logits.to(_DTYPES[case["dtype"]]),
                bias=_randn((E,), g, scale=0.1) if case["bias"] else None, ids=_ints((T, k)),
                weights=torch.zeros((T, k), device="cuda"), starts=_ints(E + 1),
                order=_ints(T * k), where=_ints((T, k)))


def _activations(T, K, g, dtype):
    """Rows of unlike size with a few channels far larger than the others."""
    x = torch.randn((T, K), device="cuda", generator=g)
    x *= torch.exp(0.3 * _randn((T, 1), g))
    x *= torch.where(_rand((1, K), g) < 0.004, 12.0, 1.0)
    return x.to(dtype)


def _prepare_quantize(case, g):
    T, K = case["T"], case["K"]
    return dict(case=case, x=_activations(T, K, g, _DTYPES[case["dtype"]]),
                codes=torch.zeros((T, K), device="cuda", dtype=_E4M3),
                scales=torch.zeros((T, K // 128), device="cuda"))


def _e4m3_weights(E, K, N, g):
    """Permuted codes [E][N][K] and the scales of 128 x 128 blocks."""
    codes = torch.empty((E, N * K), device="cuda", dtype=_E4M3)
    for e in range(E):
        codes[e] = (torch.randn(N * K, device="cuda", generator=g) * 110.0).clamp_(
            -448.0, 448.0).to(_E4M3)
    scales = torch.exp(0.3 * _randn((E, -(-N // 128), K // 128), g)) * (K ** -0.5 / 110.0)
    return codes.view(E, N, K), scales


def _prepare_dense(case, g):
    M, K, N = case["M"], case["K"], case["N"]
    dtype = _DTYPES[case["dtype"]]
    a, sa = _quantise(_activations(M, K, g, dtype))
    b, sb = _e4m3_weights(1, K, N, g)
    # the work buffer that a program keeps, zero-filled once; this size covers every case
    return dict(case=case, a=a, sa=sa, b=b[0], sb=sb[0],
                c=torch.zeros((M, N), device="cuda", dtype=dtype),
                workspace=torch.zeros(1 << 28, device="cuda", dtype=torch.uint8))


def _prepare_experts(case, g):
    T, E, k, K, N, W = (case["T"], case["E"], case["k"], case["K"], case["N"], _columns(case))
    dtype = _DTYPES[case["dtype"]]
    R = T * k
    # each token's experts, some asked for more than others; with `elsewhere`
    # as many experts again are held by another device
    score = _randn((T, E * (2 if case["elsewhere"] else 1)), g)
    score += _randn((1, score.shape[1]), g, scale=0.4)
    weights, ids = score.topk(k, dim=-1)
    ids = torch.where(ids < E, ids, E).flatten()
    order = ids.argsort(stable=True)
    where = torch.empty_like(order)
    where[order] = torch.arange(R, device="cuda")
    where = torch.where(ids < E, where, -1)
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    starts = torch.zeros(E + 1, device="cuda", dtype=torch.int64)
    starts[1:] = counts.cumsum(0)
    up = case["part"] == "up"
    s = dict(case=case, order=order.int() if up else None, starts=starts.int(),
             most=int(counts.max()), y=torch.zeros((R, N), device="cuda", dtype=dtype))
    if not up:
        s.update(where=where.int().view(T, k), weights=weights.softmax(-1),
                 out=torch.zeros((T, N), device="cuda", dtype=dtype))
    x = _activations(T if up else R, K, g, dtype)
    if case["form"] == "w8a8":
        s["a"], s["sa"] = _quantise(x)
        s["b"], s["sb"] = _e4m3_weights(E, K, W, g)
    else:
        s["a"] = x
        s["b"] = torch.randint(-2 ** 31, 2 ** 31, (E, K * W // 8), device="cuda", generator=g,
                               dtype=torch.int32)
        s["sb"] = ((0.5 + _rand((E, K // case["group"], W), g)) * (K ** -0.5 / 4.6)).to(dtype)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_route(s):
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    x = s["logits"].double()
    if case["score"] == "softmax":
        p = (x - x.amax(-1, keepdim=True)).exp()
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1.0 / (1.0 + (-x).exp())
    c = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        best = c.view(T, G, E // G).sort(dim=-1, descending=True).values[..., :case["group_best"]]
        kept = best.sum(-1).sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros((T, G), device=x.device, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, -math.inf)
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    flat = ids.flatten()
    order = flat.argsort(stable=True)
    where = torch.empty_like(order)
    where[order] = torch.arange(T * k, device=x.device)
    starts = torch.searchsorted(flat[order], torch.arange(E + 1, device=x.device))
    return [ids.int(), (w * case["scale"]).float(), starts.int(), order.int(),
            where.int().view(T, k)]


def _quantise(x):
    """16-bit rows -> e4m3 codes and FP32 scales of blocks of 128."""
    b = x.float().unflatten(-1, (-1, 128))
    scale = (b.abs().amax(-1, keepdim=True) / 448.0).clamp(min=2.0 ** -126)
    return (b * (1.0 / scale)).to(_E4M3).flatten(-2), scale.squeeze(-1)


def _plain_quantize(s):
    return _quantise(s["x"])


def _dequantise(a, sa):
    return (a.float().unflatten(-1, (-1, 128)) * sa[..., None]).flatten(-2)


def _e4m3_values(b, sb):
    """Permuted e4m3 weights [E][N][K] with block scales -> FP32 [E][K][N]."""
    E, N, K = b.shape
    w = b.view(E, N // 16, K // 128, 2, 4, 16, 16).float()
    # [E][n16][kb][half][quarter][column][i] -> [E][kb][half][quarter][i][n16][column]
    w = w.permute(0, 2, 3, 4, 6, 1, 5).reshape(E, K // 128, 128, N)
    scale = sb.transpose(1, 2).repeat_interleave(128, 2)[..., :N]
    return (w * scale[:, :, None]).view(E, K, N)


def _int4_values(b, sb, K):
    """Permuted 4-bit weights with group scales [E][groups][N] -> FP32 [E][K][N]."""
    E, G, N = sb.shape
    shift = torch.tensor([4 * n for n in _NIBBLE], device=b.device, dtype=torch.int32)
    q = (b.view(E, N // 16, K // 128, 4, 16, 4, 1) >> shift) & 15
    # [E][n16][kb][quarter][column][word][i] -> [E][kb][word][quarter][i][n16][column]
    q = q.permute(0, 2, 5, 3, 6, 1, 4).reshape(E, G, K // G, N).float() - 8.0
    return (q * sb.float()[:, :, None]).view(E, K, N)


def _plain_dense(s):
    w = _e4m3_values(s["b"][None], s["sb"][None])[0]
    return (_dequantise(s["a"], s["sa"]) @ w).to(s["c"].dtype)


def _plain_experts(s):
    case = s["case"]
    E, K, N, R = case["E"], case["K"], case["N"], s["y"].shape[0]
    starts = s["starts"].long()
    a = _dequantise(s["a"], s["sa"]) if case["form"] == "w8a8" else s["a"].float()
    w = (_e4m3_values(s["b"], s["sb"]) if case["form"] == "w8a8"
         else _int4_values(s["b"], s["sb"], K))
    # the rows of each expert, padded to the fullest one's
    at = starts[:-1, None] + torch.arange(s["most"], device=a.device)
    at = at.clamp(max=R - 1)
    y = a[at if s["order"] is None else s["order"].long()[at] // case["k"]] @ w
    if case["part"] == "up":
        gate, up = y[..., :N], y[..., N:]
        y = gate / (1.0 + (-gate).exp()) * up
    p = torch.arange(R, device=a.device)
    e = torch.searchsorted(starts[1:], p, right=True)
    live = e < E
    e = e.clamp(max=E - 1)
    y = y[e, (p - starts[e]).clamp(max=s["most"] - 1)].to(s["y"].dtype)
    y = torch.where(live[:, None], y, 0)
    if case["part"] == "up":
        return y
    here = s["where"] >= 0
    rows = y[s["where"].long().clamp(min=0)].float()
    weights = torch.where(here, s["weights"], 0.0)
    return (rows * weights[..., None]).sum(1).to(s["y"].dtype)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_route(s):
    import weight_only_int4_gemm_amd as w4
    case = s["case"]
    w4.moe_route(s["logits"], s["bias"], s["ids"], s["weights"],
                 score=w4.MOE_SOFTMAX if case["score"] == "softmax" else w4.MOE_SIGMOID,
                 groups=case["groups"], top_groups=case["top_groups"],
                 group_best=case["group_best"], renorm=bool(case["renorm"]), scale=case["scale"])
    w4.moe_tables(s["ids"], s["starts"], s["order"], s["where"])
    return [s[x] for x in ("ids", "weights", "starts", "order", "where")]


def _own_quantize(s):
    import weight_only_int4_gemm_amd as w4
    w4.w8a8_quantize(s["x"], s["codes"], s["scales"])
    return s["codes"], s["scales"]


def _own_dense(s):
    import weight_only_int4_gemm_amd as w4
    w4.w8a8_gemm(s["a"], s["sa"], s["b"], s["sb"], s["c"], s["workspace"])
    return s["c"]


def _own_experts(s):
    import weight_only_int4_gemm_amd as w4
    case = s["case"]
    act = w4.MOE_ACT_SILU_GATE if case["part"] == "up" else w4.MOE_ACT_NONE
    if case["form"] == "w8a8":
        w4.w8a8_moe_gemm(s["a"], s["sa"], s["order"], s["starts"], s["b"], s["sb"], s["y"],
                         case["k"], act)
    else:
        w4.w4a16_moe_gemm(s["a"], s["order"], s["starts"], s["b"], s["sb"], s["y"], case["k"],
                          case["group"], act)
    if case["part"] == "up":
        return s["y"]
    w4.moe_combine(s["y"], s["where"], s["weights"], s["out"])
    return s["out"]


_PREPARE = {"route": _prepare_route, "quantize": _prepare_quantize, "dense": _prepare_dense,
            "experts": _prepare_experts}
_PLAIN = {"route": _plain_route, "quantize": _plain_quantize, "dense": _plain_dense,
          "experts": _plain_experts}
_OWN = {"route": _own_route, "quantize": _own_quantize, "dense": _own_dense,
        "experts": _own_experts}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return [None, _exact_weights(s), None, None, None]
    if case["op"] == "quantize":
        return _exact_codes(s["x"])
    if case["op"] == "dense":
        return _exact_rows(s["a"], s["sa"]) @ _exact_e4m3(s["b"], s["sb"])
    return _exact_experts(s)


def _exact_weights(s):
    """The best experts taken one by one."""
    case = s["case"]
    x = s["logits"].double()
    p = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    c = p if s["bias"] is None else p + s["bias"].double()
    G = case["groups"]
    if G > 1:
        size = case["E"] // G
        marks = torch.stack([c[:, g * size:(g + 1) * size].topk(case["group_best"]).values.sum(-1)
                             for g in range(G)], 1)
        for _ in range(G - case["top_groups"]):              # the worst groups go
            worst = marks.argmin(-1)
            marks[torch.arange(case["T"], device="cuda"), worst] = math.inf
            inside = torch.arange(case["E"], device="cuda") // size == worst[:, None]
            c = c.masked_fill(inside, -math.inf)
    w = []
    for _ in range(case["k"]):
        best = c.argmax(-1, keepdim=True)
        w.append(p.gather(1, best))
        c = c.scatter(1, best, -math.inf)
    w = torch.cat(w, 1)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return w * case["scale"]


def _exact_codes(x):
    """The nearest number of three fraction bits, exponents from -6."""
    x = x.double().view(x.shape[0], -1, 128)
    scale = x.abs().amax(-1, keepdim=True).clamp(min=448 * 2.0 ** -126) / 448
    r = x / scale
    e = torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(r / step) * step).view(x.shape[0], -1), scale.squeeze(-1)


def _exact_rows(a, sa):
    return a.double() * sa.double().repeat_interleave(128, 1)


def _exact_e4m3(b, sb):
    """One matrix [K][N], byte by byte from its address."""
    N, K = b.shape
    flat = b.view(-1).view(torch.uint8)
    k, n = torch.arange(K, device="cuda")[:, None], torch.arange(N, device="cuda")[None, :]
    lane = n % 16 + 16 * (k % 64 // 16)
    at = ((n // 16 * (K // 128) + k // 128) * 2 + k % 128 // 64) * 1024 + lane * 16 + k % 16
    return flat[at].view(_E4M3).double() * sb.double()[n // 128, k // 128]


def _exact_int4(b, sb, K, group):
    N = sb.shape[1]
    k, n = torch.arange(K, device="cuda")[:, None], torch.arange(N, device="cuda")[None, :]
    lane = n % 16 + 16 * (k % 32 // 8)
    at = ((n // 16 * (K // 128) + k // 128) * 64 + lane) * 4 + k % 128 // 32
    nibble = torch.tensor(_NIBBLE, device="cuda")[k % 8]
    return ((b[at] >> (4 * nibble)) & 15).double().sub_(8).mul_(sb.double()[k // group, n])


def _exact_experts(s):
    case = s["case"]
    N, y = case["N"], torch.zeros(s["y"].shape, device="cuda", dtype=torch.float64)
    starts = s["starts"].tolist()
    for e in range(case["E"]):
        lo, hi = starts[e], starts[e + 1]
        if lo == hi:
            continue
        rows = torch.arange(lo, hi, device="cuda")
        if s["order"] is not None:
            rows = torch.div(s["order"][lo:hi].long(), case["k"], rounding_mode="floor")
        if case["form"] == "w8a8":
            a, w = _exact_rows(s["a"][rows], s["sa"][rows]), _exact_e4m3(s["b"][e], s["sb"][e])
        else:
            a, w = s["a"][rows].double(), _exact_int4(s["b"][e], s["sb"][e], case["K"],
                                                      case["group"])
        z = torch.matmul(a, w)
        y[lo:hi] = torch.nn.functional.silu(z[:, :N]) * z[:, N:] if case["part"] == "up" else z
    if case["part"] == "up":
        return y
    out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
    for j in range(case["k"]):
        at = s["where"][:, j].long()
        out += torch.where(at >= 0, s["weights"][:, j].double(), 0.0)[:, None] * y[at.clamp(min=0)]
    return out
