"""Plain reference of the expert layers and of products in 8-bit floating point.

numpy, written from the definitions (include/w4a16_moe.h and include/w8a8.h
state them); shares no code with the HIP path.  Stored forms follow the
definition's FP32 arithmetic step by step, so they can be compared bit for
bit; routing and products are float64.
"""

from __future__ import annotations

import numpy as np

f32 = np.float32
NIBBLE_OF_CODE = (0, 4, 1, 5, 2, 6, 3, 7)


# ---------------------------------------------------------------------------
# e4m3
# ---------------------------------------------------------------------------

def e4m3_value(code):
    """The number a code byte stands for: sign, 4 exponent bits (bias 7), 3
    fraction bits; exponent 0 is subnormal, 0x7f and 0xff are NaN."""
    code = np.asarray(code, np.uint8).astype(int)
    e, m = (code >> 3) & 15, code & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    x = np.where((code & 0x7F) == 0x7F, np.nan, x)
    return np.where(code & 0x80, -x, x)


_FINITE = e4m3_value(np.arange(0x7F))           # 0 .. 448, rising


def e4m3_code(x):
    """The nearest finite code, ties to the even one, the sign of x kept."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_FINITE, a).clip(1, 0x7E)
    lo = hi - 1
    up, down = _FINITE[hi] - a, a - _FINITE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quantise(x):
    """FP32 rows [T, K] -> (codes uint8 [T, K], scales float32 [T, K / 128])."""
    b = np.asarray(x, f32).reshape(len(x), -1, 128)
    bad = ~np.isfinite(b).all(-1)
    y = np.where(bad[..., None], f32(0), b)
    scale = np.maximum(np.abs(y).max(-1) / f32(448), f32(2.0 ** -126))
    q = e4m3_code(y * (f32(1) / scale)[..., None])
    q[bad] = 0
    return q.reshape(len(x), -1), np.where(bad, f32(np.nan), scale).astype(f32)


def dequantise(q, scales):
    """float64 [T, K]."""
    return e4m3_value(q) * np.repeat(scales.astype(np.float64), 128, axis=1)


def weights8(q, scales):
    """Codes [N, K] with scales [ceil(N/128), K/128] -> float64 [N, K]."""
    s = np.repeat(np.repeat(scales.astype(np.float64), 128, 0)[:q.shape[0]], 128, 1)
    return e4m3_value(q) * s


def repack8(q):
    """Codes [N, K] -> the permuted bytes."""
    N, K = q.shape
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    at = ((n // 16 * (K // 128) + k // 128) * 2 + k % 128 // 64) * 1024 \
        + (n % 16 + 16 * (k % 64 // 16)) * 16 + k % 16
    out = np.zeros(N * K, np.uint8)
    out[at] = q
    return out


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def route(logits, bias, k, softmax=True, groups=1, top_groups=1, group_best=1, renorm=True,
          scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k]), token by token."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        live = ~np.isnan(x[t]) & (x[t] > -np.inf)
        s = np.zeros(E)
        if softmax:
            if live.any():
                top = x[t][live].max()
                if top == np.inf:
                    s[live] = x[t][live] == np.inf
                else:
                    s[live] = np.exp(x[t][live] - top)
                s /= s.sum()
        else:
            with np.errstate(over="ignore"):
                s[live] = 1.0 / (1.0 + np.exp(-x[t][live]))
        c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
        live &= ~np.isnan(c) & (c > -np.inf)
        # where the order is the logits' own, they decide
        by = x[t] if bias is None and (groups == 1 or group_best == 1) else c
        if groups > 1:
            size = E // groups
            marks = []
            for g in range(groups):
                inside = [by[e] for e in range(g * size, (g + 1) * size) if live[e]]
                best = sorted(inside, reverse=True)[:group_best]
                marks.append((-sum(best), g) if best else None)
            kept = [g for _, g in sorted(m for m in marks if m is not None)[:top_groups]]
            live &= np.isin(np.arange(E) // size, kept)
        chosen = sorted((e for e in range(E) if live[e]), key=lambda e: (-by[e], e))[:k]
        w = s[chosen]
        if renorm:
            w = w / w.sum() if len(chosen) and w.sum() > 0 else w * 0
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = w * scale
    return ids, weights


def tables(ids, E):
    """(starts [E + 1], order [T * k], where [T, k]) of a routing."""
    flat = np.asarray(ids).reshape(-1)
    order = np.full(flat.size, -1, np.int32)
    where = np.full(flat.size, -1, np.int32)
    starts = np.zeros(E + 1, np.int32)
    p = 0
    for e in range(E):
        starts[e] = p
        for i in np.flatnonzero(flat == e):
            order[p], where[i] = i, p
            p += 1
    starts[E] = p
    return starts, order, where.reshape(np.shape(ids))


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def expert_rows(A, order, starts, W, k, rows):
    """(sums, sums of magnitudes) float64 [rows, columns of W]: A [a_rows, K]
    and W [E, K, columns] in float64; rows of no expert are NaN."""
    y = np.full((rows, W.shape[2]), np.nan)
    mag = np.full(y.shape, np.nan)
    for e in range(W.shape[0]):
        p = np.arange(starts[e], starts[e + 1])
        src = p if order is None else np.asarray(order)[p] // k
        y[p] = A[src] @ W[e]
        mag[p] = np.abs(A[src]) @ np.abs(W[e])
    return y, mag


def combine(Y, where, weights):
    """float64 [T, N] of rows Y, entries of `where` outside left out."""
    out = np.zeros((len(where), Y.shape[1]))
    for t in range(len(where)):
        for j, p in enumerate(where[t]):
            if 0 <= p < len(Y):
                out[t] += float(weights[t][j]) * Y[p]
    return out
