"""Cases for the 4-bit key/value cache operators: what a decoding or prefilling
attention layer does between its two weight products.

    tables     request lengths -> page tables, slots and positions (kv4_tables)
    rope       rotary positions over one to three axes            (kv4_rope)
    append     rotate, quantise to 4 bits and store; the stored
               values are read back as the outputs    (kv4_rope_append / kv4_append,
                                                       kv4_dequant_debug)
    attention  attention over the paged 4-bit cache               (kv4_attention)

With ``own`` false, ``run`` computes an operator from elementary torch
operations in 32 bits (angles in 64); with ``own`` true it calls the library.

The cache is uint8 [pages][kv heads][page][D + 8]; each (page, head) is a run
of units of 16 tokens, 16 D + 128 bytes each:

    8 D bytes   key codes    [16 tokens][D/2], channel 2i in the low nibble of byte i
    8 D bytes   value codes  [4 groups][D/8 words][4 tokens][4 bytes]
    64 bytes    key    (scale, offset) FP16 pairs [16 tokens]
    64 bytes    value  (scale, offset) FP16 pairs [16 tokens]

A stored element is (q - 8) * scale + offset, q in 0..15.
"""

import math
import random

import torch

own = False

_DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16}
_THETA = 10000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # page tables and slots of one decode step of a large serving batch
        dict(name="tables decode 256", op="tables", B=256, max_len=4096, grow=1, ends=0, page=64),
        # a scheduler step that mixes prefill chunks, decode steps, roll-backs
        # of rejected draft tokens and requests that end
        dict(name="tables mixed 1000", op="tables", B=1000, max_len=2048, grow=160, ends=1,
             page=16),
        # query rotation of one decode step, one axis (text)
        dict(name="rope decode 64", op="rope", T=64, H=32, D=128, rot=128, axes=1, pairs=0,
             far=4096, dtype="float16"),
        # an image/video prefill: time, height and width positions
        dict(name="rope video 16384", op="rope", T=16384, H=32, D=128, rot=128, axes=3, pairs=0,
             far=1000000, dtype="bfloat16"),
        # one decode step of a grouped-query layer (8192 wide, 64 query and 8
        # key/value heads): rotate q and k, store k and v
        dict(name="append decode 32", op="append", T=32, Hq=64, H=8, D=128, rot=128, axes=1,
             pairs=0, far=4096, page=64, dtype="float16"),
        # a prefill of the same layer, positions on three axes
        dict(name="append prefill 8192", op="append", T=8192, Hq=64, H=8, D=128, rot=128, axes=3,
             pairs=0, far=100000, page=64, dtype="bfloat16"),
        # keys rotated elsewhere, heads as many as query heads (4096 wide), an odd token count
        dict(name="append stored 4001", op="append", T=4001, Hq=0, H=32, D=128, rot=0, axes=0,
             pairs=0, far=0, page=32, dtype="float16"),
        # one short conversation, one token: latency alone
        dict(name="attention decode 1x1000", op="attention", B=1, max_len=1000, nq=1, Hq=32, H=32,
             D=128, page=64, window=0, dtype="float16"),
        # a full decode batch of the 4096-wide layer: cache bandwidth
        dict(name="attention decode 64x4096", op="attention", B=64, max_len=4096, nq=1, Hq=32,
             H=32, D=128, page=64, window=0, dtype="float16"),
        # one long document, grouped heads: few rows, a long axis
        dict(name="attention decode 1x131072", op="attention", B=1, max_len=131072, nq=1, Hq=64,
             H=8, D=128, page=128, window=0, dtype="bfloat16"),
        # draft tokens verified against a sliding window, small heads
        dict(name="attention verify 24x5", op="attention", B=24, max_len=8000, nq=5, Hq=32, H=8,
             D=64, page=16, window=4096, dtype="float16"),
        # chunks of long prompts over what is stored already: matrix bound
        dict(name="attention prefill 2x2048", op="attention", B=2, max_len=8192, nq=2048, Hq=64,
             H=8, D=128, page=64, window=0, dtype="bfloat16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        case = _draw_one(rng)
        if _cost(case) <= most and _plain_bytes(case) <= 24e9:
            return case


def _plain_bytes(case):
    """About what the plain attention holds at once."""
    if case["op"] != "attention":
        return 0
    rows = case["B"] * case["max_len"]
    return 4 * (4 * rows * case["H"] * case["D"] + 3 * rows * case["nq"] * case["Hq"])


def _draw_one(rng):
    op = rng.choice(("tables", "rope", "append", "attention", "attention", "attention"))
    dtype = rng.choice(("float16", "bfloat16"))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "tables":
        return dict(op=op, B=_spread(rng, 1, 2048), max_len=_spread(rng, 256, 8192),
                    grow=rng.choice((1, 1, 4, _spread(rng, 2, 200))), ends=rng.randrange(2),
                    page=page)
    D = rng.choice((64, 128, 128, 256))
    rot = rng.choice((D, D, D // 2))
    axes = rng.choice((1, 2, 3))
    far = _spread(rng, 256, 1000000)
    if op == "rope":
        return dict(op=op, T=_spread(rng, 1, 16384), H=rng.choice((1, 4, 8, 12, 32)), D=D,
                    rot=rot, axes=axes, pairs=rng.randrange(2), far=far, dtype=dtype)
    H = rng.choice((1, 2, 4, 8, 8, 32))
    group = rng.choice((1, 1, 3, 4, 7, 8, 16))
    if op == "append":
        fused = rng.randrange(3) > 0
        return dict(op=op, T=_spread(rng, 1, 8192), Hq=H * group if fused else 0, H=H, D=D,
                    rot=rot if fused else 0, axes=axes if fused else 0,
                    pairs=rng.randrange(2) if fused else 0, far=far if fused else 0, page=page,
                    dtype=dtype)
    nq = rng.choice((1, 1, 1, _spread(rng, 2, 16), _spread(rng, 16, 2048)))
    return dict(op=op, B=_spread(rng, 1, 128), max_len=_spread(rng, max(nq, 16), 131072), nq=nq,
                Hq=H * group, H=H, D=D, page=page,
                window=rng.choice((0, 0, 0, _spread(rng, 16, 8192))), dtype=dtype)


def _lengths(case):
    """The ragged lengths of a batch: (tokens held after the call, new
    queries), the same for every seed, the first request at the maximum."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    lens, new = [], []
    for b in range(case["B"]):
        n = case["nq"] if b == 0 or case["nq"] < 16 else r.randint(case["nq"] // 2, case["nq"])
        lens.append(case["max_len"] if b == 0
                    else r.randint(max(n, case["max_len"] // 4), max(n, case["max_len"])))
        new.append(n)
    return lens, new


def _wanted(case):
    """(tokens held, tokens wanted) of each request of a scheduler step."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    held, want = [], []
    for b in range(case["B"]):
        n = r.randint(0, case["max_len"] - case["grow"])
        kind = r.random()
        if case["ends"] and kind < 0.1:
            w = 0
        elif case["ends"] and kind < 0.2:
            w = max(0, n - r.randint(0, 4))
        else:
            w = n + (case["grow"] if case["grow"] <= 4 else r.randint(1, case["grow"]))
        held.append(n)
        want.append(w)
    return held, want


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "tables":
        held, want = _wanted(case)
        p = case["page"]
        moved = sum(abs(-(-w // p) + (-h // p)) for h, w in zip(held, want))
        new = sum(max(0, w - h) for h, w in zip(held, want))
        return {"bytes": 4 * (4 * case["B"] + 2 * moved + 2 * new), "flops": 0}
    if op == "rope":
        n = case["T"] * case["H"]
        return {"bytes": 4 * n * case["D"] + 4 * case["axes"] * case["T"],
                "flops": 3 * n * case["rot"]}
    if op == "append":
        kv = case["T"] * case["H"]
        # q in and out; k and v in, stored, read back and written out
        return {"bytes": case["T"] * (4 * case["Hq"] * case["D"] + 4 * case["axes"] + 4)
                + kv * (2 * 4 * case["D"] + 2 * (case["D"] + 8)),
                "flops": 3 * case["T"] * (case["Hq"] + case["H"]) * case["rot"]
                + 12 * kv * case["D"]}
    lens, new = _lengths(case)
    w = case["window"] or case["max_len"] + 1
    cached = sum(min(n, w + m - 1) for n, m in zip(lens, new))
    seen = sum(_keys_seen(n, m, w) for n, m in zip(lens, new))
    rows = sum(new) * case["Hq"]
    return {"bytes": cached * case["H"] * (case["D"] + 8) + rows * (4 * case["D"] + 4),
            "flops": 4 * case["D"] * case["Hq"] * seen}


def _keys_seen(n, m, w):
    """Keys that m causal queries at the end of n tokens see within w."""
    full = max(0, min(m, n - w))               # queries whose window is whole
    rest = m - full                            # the others see all before them
    first = n - m + 1
    return full * w + rest * first + rest * (rest - 1) // 2


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sections(rot, axes):
    """Frequency pairs of each axis: about a quarter to time, the rest to
    height and width."""
    half = rot // 2
    if axes <= 1:
        return (half,)
    if axes == 2:
        return (half // 2, half - half // 2)
    first = half // 4
    return (first, (half - first) // 2, half - first - (half - first) // 2)


def _positions(case, g):
    """Positions in reading order on every axis, ending near case["far"]."""
    T, axes, far = case["T"], case["axes"], case["far"]
    start = max(0, far - T)
    pos = torch.arange(start, start + T, device="cuda", dtype=torch.int32).repeat(axes, 1)
    jitter = torch.randint(0, 64, (axes, T), device="cuda", generator=g, dtype=torch.int32)
    jitter[0] = 0
    return (pos + jitter).contiguous()


def _inv_freq(rot):
    i = torch.arange(0, rot, 2, device="cuda", dtype=torch.float64)
    return _THETA ** (-i / rot)


def _randn(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return _PREPARE[case["op"]](case, g)


def _prepare_tables(case, g):
    held, want = _wanted(case)
    B, page = case["B"], case["page"]
    lens = torch.tensor(held, device="cuda", dtype=torch.int32)
    width = -(-case["max_len"] // page) + 1
    used = [-(-n // page) for n in held]
    spare = sum(max(0, -(-w // page) - u) for w, u in zip(want, used)) + B
    pages = sum(used) + spare
    ids = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    table = torch.full((B, width), -1, device="cuda", dtype=torch.int32)
    cols = torch.arange(width, device="cuda")
    held_pages = (lens + page - 1) // page
    table[cols[None, :] < held_pages[:, None]] = ids[: sum(used)]
    # the queue of free pages starts anywhere in its ring
    head = int(torch.randint(0, pages, (1,), device="cuda", generator=g))
    ring = torch.full((pages,), -1, device="cuda", dtype=torch.int32)
    ring[(head + torch.arange(spare, device="cuda")) % pages] = ids[sum(used):]
    new = sum(max(0, w - h) for h, w in zip(held, want))
    capacity = -(-max(1, new) // 64) * 64
    z = lambda n: torch.zeros(n, device="cuda", dtype=torch.int32)  # noqa: E731
    return dict(case=case, lens=lens, want=torch.tensor(want, device="cuda", dtype=torch.int32),
                table=table, ring=ring,
                state=torch.tensor([head, spare, 0, 0], device="cuda", dtype=torch.int32),
                lens_out=z(B), state_out=z(4), q_start=z(B + 1), slots=z(capacity),
                positions=z(capacity))


def _prepare_rope(case, g):
    dtype = _DTYPES[case["dtype"]]
    x = _randn((case["T"], case["H"], case["D"]), dtype, g)
    return dict(case=case, x=x, y=torch.empty_like(x), positions=_positions(case, g),
                inv_freq=_inv_freq(case["rot"]), sections=_sections(case["rot"], case["axes"]))


def _prepare_append(case, g):
    T, Hq, H, D, page = (case[k] for k in ("T", "Hq", "H", "D", "page"))
    dtype = _DTYPES[case["dtype"]]
    # the three parts of one fused product's output
    qkv = _randn((T, Hq + 2 * H, D), dtype, g)
    spread = torch.exp(0.5 * torch.randn((1, H, D), device="cuda", generator=g))
    qkv[:, Hq:Hq + H] = (qkv[:, Hq:Hq + H] * spread).to(dtype)
    pages = -(-T // page) + 2
    order = torch.randperm(pages, device="cuda", generator=g)
    at = torch.arange(T, device="cuda") + page // 3
    slots = (order[at // page] * page + at % page).to(torch.int32)
    s = dict(case=case, q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H], v=qkv[:, Hq + H:], slots=slots,
             cache=torch.zeros((pages, H, page, D + 8), device="cuda", dtype=torch.uint8),
             k_out=torch.empty((T, H, D), device="cuda", dtype=dtype),
             v_out=torch.empty((T, H, D), device="cuda", dtype=dtype))
    if Hq:
        s.update(q_out=torch.empty((T, Hq, D), device="cuda", dtype=dtype),
                 positions=_positions(case, g), inv_freq=_inv_freq(case["rot"]),
                 sections=_sections(case["rot"], case["axes"]))
    return s


def _prepare_attention(case, g):
    B, Hq, H, D, page = (case[k] for k in ("B", "Hq", "H", "D", "page"))
    dtype = _DTYPES[case["dtype"]]
    lens, new = _lengths(case)
    width = -(-case["max_len"] // page)
    used = [-(-n // page) for n in lens]
    order = torch.randperm(sum(used) + 1, device="cuda", generator=g)
    table = torch.full((B, width), -1, device="cuda", dtype=torch.int32)
    used_t = torch.tensor(used, device="cuda")
    table[torch.arange(width, device="cuda")[None, :] < used_t[:, None]] = \
        order[: sum(used)].to(torch.int32)
    cache = torch.zeros((sum(used) + 1, H, page, D + 8), device="cuda", dtype=torch.uint8)
    # keys with channels of unlike size, values without, as projections give them
    spread = torch.exp(0.4 * torch.randn((1, H, D), device="cuda", generator=g))
    total = sum(lens)
    ends = torch.tensor(lens, device="cuda").cumsum(0)
    step = max(1, (1 << 27) // (H * D))
    for t0 in range(0, total, step):
        t = torch.arange(t0, min(total, t0 + step), device="cuda")
        b = torch.searchsorted(ends, t, right=True)
        at = t - (ends[b] - torch.tensor(lens, device="cuda")[b])
        slots = table[b, at // page].long() * page + at % page
        k = torch.randn((t.numel(), H, D), device="cuda", generator=g) * spread
        v = torch.randn((t.numel(), H, D), device="cuda", generator=g)
        _store(cache, slots, k.to(dtype).float(), v.to(dtype).float())
    T = sum(new)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = dict(case=case, q=_randn((T, Hq, D), dtype, g, 1.3), cache=cache, table=table,
             lens=torch.tensor(lens, device="cuda", dtype=torch.int32),
             q_start=torch.tensor(starts, device="cuda", dtype=torch.int32),
             o=torch.empty((T, Hq, D), device="cuda", dtype=dtype),
             lse=torch.empty((T, Hq), device="cuda", dtype=torch.float32), scale=D ** -0.5)
    # the work buffer that a program keeps beside its cache, zero-filled once;
    # this size covers every case
    s["workspace"] = torch.zeros(1 << 28, device="cuda", dtype=torch.uint8)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _unit_views(cache):
    """Key codes, value codes and parameters of a cache, as strided views."""
    P, H, page, D8 = cache.shape
    D = D8 - 8
    u = cache.view(P, H, page // 16, 16 * D8)
    k = u[..., : 8 * D].unflatten(-1, (16, D // 2))
    v = u[..., 8 * D: 16 * D].unflatten(-1, (4, D // 8, 4, 4))
    par = u[..., 16 * D:].view(torch.float16).unflatten(-1, (2, 16, 2))
    return k, v, par


def _quantise(x):
    """FP32 rows [..., D] -> codes and their FP16 (scale, offset)."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) * (1.0 / 15.0)).half().float()
    z = (lo + 8.0 * s).half().float()
    r = torch.where(s > 0, 1.0 / s, torch.zeros_like(s))
    q = (torch.round((x - z) * r) + 8.0).clamp(0.0, 15.0).to(torch.uint8)
    return q, torch.cat((s, z), -1).half()


def _store(cache, slots, k, v):
    kc, vc, par = _unit_views(cache)
    page = cache.shape[2]
    pg, at = slots // page, slots % page
    u, r = at // 16, at % 16
    q, p = _quantise(k)
    kc[pg, :, u, r] = q[..., 0::2] | (q[..., 1::2] << 4)
    par[pg, :, u, 0, r] = p
    q, p = _quantise(v)
    q = q[..., 0::2] | (q[..., 1::2] << 4)
    vc[pg, :, u, r // 4, :, r % 4] = q.unflatten(-1, (-1, 4))
    par[pg, :, u, 1, r] = p


def _decode(b, p):
    """Code bytes [..., D/2] and their (scale, offset) [..., 2] -> FP32 [..., D]."""
    q = torch.stack((b & 15, b >> 4), -1).flatten(-2).float()
    p = p.float()
    return (q - 8.0) * p[..., :1] + p[..., 1:]


def _rotate(x, positions, inv_freq, sections, pairs):
    """Rotary positions of [T, H, D] in 32 bits, the angles in 64."""
    axis = torch.repeat_interleave(
        torch.arange(len(sections), device=x.device),
        torch.tensor(sections, device=x.device), output_size=sum(sections))
    angle = positions.double()[axis].t() * inv_freq          # [T, rot / 2]
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    rot = 2 * sum(sections)
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., : rot // 2],
                                                              x[..., rot // 2: rot])
    ra, rb = a * c - b * s, b * c + a * s
    y = torch.stack((ra, rb), -1).flatten(-2) if pairs else torch.cat((ra, rb), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_tables(s):
    lens, want, table, ring, state = (s[k].long() for k in ("lens", "want", "table", "ring",
                                                            "state"))
    page, (B, width), P = s["case"]["page"], table.shape, ring.numel()
    head, count = state[0], state[1]
    old, new = (lens + page - 1) // page, (want + page - 1) // page
    over = new > width
    need = torch.where(over, 0, new - old).clamp(min=0)
    free = torch.where(over, 0, old - new).clamp(min=0)
    upto = need.cumsum(0)
    served = ~over & ((need == 0) | (upto <= count))
    taken = torch.where(served & (need > 0), upto, 0).amax()
    col = torch.arange(width, device=table.device)[None, :]
    fresh = served[:, None] & (col >= old[:, None]) & (col < new[:, None])
    place = (head + (upto - need)[:, None] + col - old[:, None]) % P
    table = torch.where(fresh, ring[place], table)
    gone = (col >= new[:, None]) & (col < old[:, None]) & ~over[:, None]
    to = (head + count + (free.cumsum(0) - free)[:, None] + col - new[:, None]) % P
    ring = torch.cat((ring, ring[:1]))
    ring.scatter_(0, torch.where(gone, to, P).flatten(), table.flatten())
    grown = (want - lens).clamp(min=0)
    q_start = torch.cat((grown[:1] * 0, grown.cumsum(0)))
    t = torch.arange(s["slots"].numel(), device=table.device)
    b = torch.searchsorted(q_start[1:], t, right=True).clamp(max=B - 1)
    live = t < q_start[-1]
    pos = torch.where(live, lens[b] + t - q_start[b], 0)
    entry = table[b, (pos // page).clamp(max=width - 1)]
    slots = torch.where(live & served[b], entry * page + pos % page, -1)
    state = torch.stack(((head + taken) % P, count - taken + free.sum(), (~served).sum(),
                         head * 0))
    out = (torch.where(served, want, lens), table, ring[:P], state, q_start, slots, pos)
    return [x.int() for x in out]


def _plain_rope(s):
    y = _rotate(s["x"], s["positions"], s["inv_freq"], s["sections"], s["case"]["pairs"])
    return y.to(s["x"].dtype)


def _plain_append(s):
    case, dtype = s["case"], s["k"].dtype
    k, out = s["k"].float(), []
    if case["Hq"]:
        rot = (s["positions"], s["inv_freq"], s["sections"], case["pairs"])
        out = [_rotate(s["q"], *rot).to(dtype)]
        k = _rotate(k, *rot)
    slots, page = s["slots"].long(), case["page"]
    _store(s["cache"], slots, k, s["v"].float())
    kc, vc, par = _unit_views(s["cache"])
    pg, at = slots // page, slots % page
    u, r = at // 16, at % 16
    out.append(_decode(kc[pg, :, u, r], par[pg, :, u, 0, r]).to(dtype))
    out.append(_decode(vc[pg, :, u, r // 4, :, r % 4].flatten(-2), par[pg, :, u, 1, r]).to(dtype))
    return out


def _plain_attention(s):
    case, cache = s["case"], s["cache"]
    B, Hq, H, D, nq = (case[k] for k in ("B", "Hq", "H", "D", "nq"))
    L = s["table"].shape[1] * case["page"]
    kc, vc, par = _unit_views(cache[s["table"].long().clamp(min=0)].flatten(0, 1))
    par = par.unflatten(0, (B, -1)).transpose(1, 2)         # [B, H, pages, units, 2, 16, 2]
    kc = kc.unflatten(0, (B, -1)).transpose(1, 2).reshape(B, H, L, D // 2)
    k = _decode(kc, par[..., 0, :, :].reshape(B, H, L, 2))
    vc = vc.unflatten(0, (B, -1)).transpose(1, 2).transpose(-3, -2).reshape(B, H, L, D // 2)
    v = _decode(vc, par[..., 1, :, :].reshape(B, H, L, 2))
    lens, starts = s["lens"].long(), s["q_start"].long()
    n = starts[1:] - starts[:-1]
    i = torch.arange(nq, device=cache.device)
    q = s["q"][(starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()
    q = q.view(B, nq, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    j = torch.arange(L, device=cache.device)
    at = (lens - n)[:, None] + i                             # a query's own position
    seen = (j <= at[..., None]) & (j < lens[:, None, None])
    if case["window"]:
        seen &= j > at[..., None] - case["window"]
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0.0)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, H, Hq // H, nq, L)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    d = p.sum(-1, keepdim=True)
    o = (p.view(B, H, -1, L) @ v).view(B, H, Hq // H, nq, D)
    o = torch.where(d > 0, o / d, 0.0).permute(0, 3, 1, 2, 4).reshape(B, nq, Hq, D)
    lse = (m + d.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, nq, Hq)
    t = torch.arange(s["q"].shape[0], device=cache.device)
    b = torch.searchsorted(starts[1:], t, right=True)
    return o[b, t - starts[b]].to(s["q"].dtype), lse[b, t - starts[b]]


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own_tables(s):
    import weight_only_int4_gemm_amd as w4
    w4.kv4_tables(s["lens"], s["want"], s["table"], s["ring"], s["state"], s["lens_out"],
                  s["state_out"], s["q_start"], s["slots"], s["positions"], s["case"]["page"])
    return [s[k] for k in ("lens_out", "table", "ring", "state_out", "q_start", "slots",
                           "positions")]


def _own_rope(s):
    import weight_only_int4_gemm_amd as w4
    w4.kv4_rope(s["x"], s["y"], s["positions"], s["inv_freq"], s["sections"], s["case"]["pairs"])
    return s["y"]


def _own_append(s):
    import weight_only_int4_gemm_amd as w4
    out = [s["k_out"], s["v_out"]]
    if s["case"]["Hq"]:
        w4.kv4_rope_append(s["q"], s["k"], s["v"], s["q_out"], s["positions"], s["inv_freq"],
                           s["sections"], s["case"]["pairs"], s["slots"], s["cache"])
        out = [s["q_out"]] + out
    else:
        w4.kv4_append(s["k"], s["v"], s["slots"], s["cache"])
    w4.kv4_dequant_debug(s["slots"], s["cache"], s["k_out"], s["v_out"])
    return out


def _own_attention(s):
    import weight_only_int4_gemm_amd as w4
    case = s["case"]
    w4.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["q_start"], s["o"], s["lse"],
                     s["scale"], case["window"], case["nq"], case["max_len"], s["workspace"])
    return s["o"], s["lse"]


_PREPARE = {"tables": _prepare_tables, "rope": _prepare_rope, "append": _prepare_append,
            "attention": _prepare_attention}
_PLAIN = {"tables": _plain_tables, "rope": _plain_rope, "append": _plain_append,
          "attention": _plain_attention}
_OWN = {"tables": _own_tables, "rope": _own_rope, "append": _own_append,
        "attention": _own_attention}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None                                          # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s, s["x"])
    if case["op"] == "append":
        out, k = [], s["k"].double()
        if case["Hq"]:
            out.append(_exact_rotation(s, s["q"]))
            k = _exact_rotation(s, k)
        return out + [_exact_four_bits(k), _exact_four_bits(s["v"].double())]
    return _exact_attention(s)


def _exact_rotation(s, x):
    """Each pair as a complex number times exp(i angle)."""
    case = s["case"]
    half = case["rot"] // 2
    of = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    freq = _THETA ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / case["rot"])
    angle = torch.stack([s["positions"][a].double() for a in of], 1) * freq
    x = x.double()
    ia = torch.arange(half, device="cuda") * (2 if case["pairs"] else 1)
    ib = ia + (1 if case["pairs"] else half)
    turned = torch.complex(x[..., ia], x[..., ib]) * torch.polar(torch.ones_like(angle),
                                                                 angle)[:, None]
    y = x.clone()
    y[..., ia], y[..., ib] = turned.real, turned.imag
    return y


def _exact_four_bits(x):
    """The nearest of the sixteen values of each row's scale and offset."""
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    scale = ((high - low) / 15).half().double()
    offset = (low + 8 * scale).half().double()
    steps = torch.where(scale > 0, (x - offset) / scale, torch.zeros_like(x))
    return torch.clamp(torch.round(steps), -8, 7) * scale + offset


def _exact_attention(s):
    """Request by request: words and parameters by their addresses."""
    case = s["case"]
    H, D, page = case["H"], case["D"], case["page"]
    group, unit = case["Hq"] // H, 16 * (D + 8)
    words = s["cache"].view(-1).view(torch.int32)
    halves = s["cache"].view(-1).view(torch.float16)
    lens, starts = s["lens"].tolist(), s["q_start"].tolist()
    out = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(s["q"].shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    shift = torch.arange(0, 32, 4, device="cuda")
    word = torch.arange(D // 8, device="cuda")
    for b in range(case["B"]):
        n, t0, t1 = lens[b], starts[b], starts[b + 1]
        j = torch.arange(n, device="cuda")
        at = torch.arange(n - (t1 - t0), n, device="cuda")
        hide = j[None, :] > at[:, None]
        if case["window"]:
            hide |= j[None, :] <= at[:, None] - case["window"]
        for h in range(H):
            base = ((s["table"][b, j // page].long() * H + h) * (page // 16) + j % page // 16) * unit
            r = j % 16
            kw = words[(base // 4 + r * (D // 8))[:, None] + word]
            vw = words[(base // 4 + 2 * D + r // 4 * (D // 2) + r % 4)[:, None] + 4 * word]
            p = base // 2 + 8 * D + 2 * r
            k = ((kw[..., None] >> shift) & 15).flatten(1).double() - 8
            k = k * halves[p].double()[:, None] + halves[p + 1].double()[:, None]
            v = ((vw[..., None] >> shift) & 15).flatten(1).double() - 8
            v = v * halves[p + 32].double()[:, None] + halves[p + 33].double()[:, None]
            q = s["q"][t0:t1, h * group:(h + 1) * group].double().transpose(0, 1)
            x = torch.matmul(q, k.t().contiguous()) * s["scale"]
            x = x.masked_fill(hide, -math.inf)
            out[t0:t1, h * group:(h + 1) * group] = torch.matmul(x.softmax(-1), v).transpose(0, 1)
            lse[t0:t1, h * group:(h + 1) * group] = x.logsumexp(-1).transpose(0, 1)
    return out, lse
