"""Plain reference of the paged 4-bit key/value cache operators.

numpy, written from the definitions (include/w4a16_kv4.h states them); shares
no code with the HIP path.  Stored forms follow the definition's FP32
arithmetic step by step, so they can be compared bit for bit; rotations and
attention are float64.
"""

from __future__ import annotations

import numpy as np

f32 = np.float32


def round_half(x):
    """FP32 -> FP16, half to even, as uint16 bits."""
    with np.errstate(over="ignore"):
        return np.asarray(x, f32).astype(np.float16).view(np.uint16)


def quantise(x):
    """Rows [..., D] -> (codes uint8 [..., D], params uint16 [..., 2])."""
    x = np.asarray(x, f32)
    bad = ~np.isfinite(x).all(-1)
    y = np.where(bad[..., None], f32(0), x)
    lo, hi = y.min(-1), y.max(-1)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        s = np.minimum((hi - lo) * (f32(1) / f32(15)), f32(65504)).astype(np.float16)
        s32 = s.astype(f32)
        z = np.clip(lo + f32(8) * s32, f32(-65504), f32(65504)).astype(np.float16)
        inv = np.where(s32 > 0, f32(1) / s32, f32(0)).astype(f32)
        q = np.rint((y - z.astype(f32)[..., None]) * inv[..., None]) + f32(8)
    q = np.clip(q, 0, 15).astype(np.uint8)
    q[bad] = 8
    par = np.stack((s.view(np.uint16), z.view(np.uint16)), -1)
    par[bad] = 0x7E00
    return q, par


def unit_bytes(D):
    return 16 * D + 128


def _unit(pages, heads, page, D, slot, head):
    """Byte offset of the unit that holds `slot`, and the token's row in it."""
    pid, at = divmod(int(slot), page)
    return ((pid * heads + head) * (page // 16) + at // 16) * unit_bytes(D), at % 16


def store(cache, slots, K, V):
    """Append FP32 rows K, V [T, heads, D] to ``cache`` uint8 [pages, heads,
    page, D + 8] in place."""
    pages, heads, page, d8 = cache.shape
    D = d8 - 8
    flat = cache.reshape(-1)
    for X, values in ((K, False), (V, True)):
        codes, params = quantise(X)
        for t, slot in enumerate(slots):
            if not 0 <= slot < pages * page:
                continue
            for h in range(heads):
                base, r = _unit(pages, heads, page, D, slot, h)
                q = codes[t, h].astype(np.uint8)
                b = (q[0::2] | (q[1::2] << 4)).reshape(D // 8, 4)   # bytes of each word
                for w in range(D // 8):
                    at = (8 * D + ((r // 4 * (D // 8) + w) * 4 + r % 4) * 4 if values
                          else r * (D // 2) + 4 * w)
                    flat[base + at: base + at + 4] = b[w]
                at = base + 16 * D + (64 if values else 0) + 4 * r
                flat[at: at + 4] = params[t, h].astype("<u2").view(np.uint8)


def load(cache, slots):
    """(codes, scale, offset) of keys and of values at ``slots``: codes
    float64 [T, heads, D] centred on 8, scale and offset float64 [T, heads]."""
    pages, heads, page, d8 = cache.shape
    D = d8 - 8
    flat = cache.reshape(-1)
    out = []
    for values in (False, True):
        c = np.zeros((len(slots), heads, D))
        s = np.zeros((len(slots), heads))
        z = np.zeros((len(slots), heads))
        for t, slot in enumerate(slots):
            if not 0 <= slot < pages * page:
                continue
            for h in range(heads):
                base, r = _unit(pages, heads, page, D, slot, h)
                if values:
                    codes = flat[base + 8 * D: base + 16 * D].view("<u4").reshape(4, D // 8, 4)
                    words = codes[r // 4, :, r % 4]
                else:
                    words = flat[base: base + 8 * D].view("<u4").reshape(16, D // 8)[r]
                for k in range(8):
                    c[t, h, k::8] = ((words >> np.uint32(4 * k)) & np.uint32(15)).astype(float) - 8
                at = base + 16 * D + (64 if values else 0) + 4 * r
                s[t, h], z[t, h] = flat[at: at + 4].view("<f2").astype(float)
        out.append((c, s, z))
    return out


def values_of(part):
    c, s, z = part
    return c * s[..., None] + z[..., None]


def rope(x, positions, inv_freq, sections, pairs):
    """float64 rotation of [T, H, D]; positions [axes, T]."""
    x = np.asarray(x, np.float64)
    half = sum(sections)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = np.asarray(positions, np.float64)[axis].T * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def attention(q, cache, table, lens, q_start, scale, window=0, max_q=None):
    """float64 attention.  Returns (o, lse, weight, size, floor, reach) over
    rows [T, Hq]: besides the results, per element the sums that error bounds
    are made of: ``weight`` = sum p s |c - 8|, ``size`` = sum p (15 s + |z|)
    and ``floor`` = 8 n max(p s) for n keys, and per row ``reach`` = the
    largest magnitude that a score is summed from.  Rows of no request are
    NaN."""
    pages, H, page, d8 = cache.shape
    D = d8 - 8
    q = np.asarray(q, np.float64)
    T, Hq, _ = q.shape
    group = Hq // H
    B, width = table.shape
    o = np.full(q.shape, np.nan)
    weight, size, floor = (np.zeros(q.shape) for _ in range(3))
    lse, reach = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for b in range(B):
        n = min(max(int(lens[b]), 0), width * page)
        t0, t1 = (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))
        j = np.arange(n)
        ids = table[b, j // page].astype(np.int64)
        there = (ids >= 0) & (ids < pages)
        slots = np.where(there, ids * page + j % page, -1)
        (kc, ks, kz), (vc, vs, vz) = load(cache, slots)
        for t in range(t0, t1):
            if max_q is not None and t - t0 >= max_q:
                continue
            pos = n - (t1 - t0) + (t - t0)
            see = there & (j <= pos)
            if window:
                see &= j > pos - window
            for h in range(Hq):
                g = h // group
                if not see.any():
                    o[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                k = kc[see, g] * ks[see, g, None] + kz[see, g, None]
                x = scale * (k @ q[t, h])
                m = x.max()
                p = np.exp(x - m)
                lse[t, h] = m + np.log(p.sum())
                p /= p.sum()
                o[t, h] = p @ (vc[see, g] * vs[see, g, None] + vz[see, g, None])
                weight[t, h] = (p * vs[see, g]) @ np.abs(vc[see, g])
                floor[t, h] = 8 * len(p) * (p * vs[see, g]).max()
                size[t, h] = (p * (15 * vs[see, g] + np.abs(vz[see, g]))).sum()
                reach[t, h] = (scale * np.abs(q[t, h]).sum()
                               * (23 * ks[see, g] + np.abs(kz[see, g])).max())
    return o, lse, weight, size, floor, reach


def tables(lens, want, table, ring, state, capacity, page):
    """One scheduler step, request by request.  Returns (lens_out, table, ring,
    state_out, q_start, slots, positions); the inputs are left alone."""
    table, ring = np.array(table), np.array(ring)
    B, width = table.shape
    pages = len(ring)
    head, count = int(state[0]), int(state[1])
    before = np.array(table)
    lens_out, q_start = [], [0]
    slots, positions = [-1] * capacity, [0] * capacity
    wanted = taken = returned = refused = 0
    ends = 0                                # new tokens so far, refused or not
    for b in range(B):
        n = min(max(int(lens[b]), 0), width * page)
        w = max(int(want[b]), 0)
        old, new = -(-n // page), -(-w // page)
        grown = max(0, w - n)
        ends += grown
        ok = new <= width and (grown == 0 or ends <= capacity)
        if ok and new > old:
            ids = []
            if wanted + new - old <= count:
                ids = [int(ring[(head + wanted + i) % pages]) for i in range(new - old)]
                table[b, old:new] = ids
            wanted += new - old
            ok = bool(ids)
            if ok:
                taken = wanted
        refused += not ok
        if new < old:
            for i in range(new, old):
                ring[(head + count + returned) % pages] = before[b, i]
                returned += 1
        for i in range(grown):
            t = q_start[-1] + i
            if t >= capacity:
                break
            positions[t] = n + i
            if ok:
                pid = int(table[b, (n + i) // page])
                if 0 <= pid < pages:
                    slots[t] = pid * page + (n + i) % page
        q_start.append(min(capacity, ends))
        lens_out.append(w if ok else n)
    state_out = [(head + taken) % pages, min(pages, count - taken + returned), refused, 0]
    return (np.array(lens_out, np.int32), table, ring, np.array(state_out, np.int32),
            np.array(q_start, np.int32), np.array(slots, np.int32),
            np.array(positions, np.int32))
