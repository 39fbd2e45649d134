"""Float64 reference of the 4-bit key/value cache and of the key mass.

The format: a row of D dims is D e2m1 codes (sign, two exponent bits with bias 1,
one fraction bit) and one e4m3 scale (four exponent bits with bias 7, three
fraction bits, no infinity, 0x7F is NaN) for each 16 dims; a value is
code * scale * tensor scale. Rounding is to nearest, ties to the even code, by
comparing exact distances. Loops and explicit score matrices: small sizes only.
"""
from __future__ import annotations

import numpy as np

BLOCK = 16


def e2m1_value(code: int) -> float:
    e, m = (code >> 1) & 3, code & 1
    x = (1 + m / 2) * 2.0 ** (e - 1) if e else m / 2
    return -x if code & 8 else x


def e4m3_value(code: int) -> float:
    if code & 0x7F == 0x7F:
        return float("nan")
    e, m = (code >> 3) & 15, code & 7
    x = (1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9
    return -x if code & 0x80 else x


E2M1 = np.array([e2m1_value(c) for c in range(16)])
E4M3 = np.array([e4m3_value(c) for c in range(256)])


def nearest_even(x: float, unit: float, values) -> int:
    """Index of the value v in `values` (ascending) with x nearest to v * unit;
    between two equally near the even index; beyond the last, the last."""
    if x >= values[-1] * unit:          # also where the distances would all round to x
        return len(values) - 1
    best = 0
    for i in range(1, len(values)):
        near, far = abs(x - values[i] * unit), abs(x - values[best] * unit)
        if near < far or (near == far and i % 2 == 0):
            best = i
    return best


def quantise_block(x, ts: float):
    """(codes, scale code) of up to 16 values."""
    x = np.asarray(x, dtype=np.float64)
    if not np.isfinite(x).all():
        return [0] * len(x), 0x7F
    # nearest scale to max / (6 ts): distances of max to scale * 6 ts
    s = nearest_even(float(np.abs(x).max()), 6.0 * ts, E4M3[:127])
    d = E4M3[s] * ts
    return [(8 if np.signbit(v) else 0) | (nearest_even(abs(float(v)), d, E2M1[:8]) if d > 0 else 0) for v in x], s


def quantise_row(x, ts: float):
    """(packed codes uint8 [D / 2], scales uint8 [ceil(D / 16)])."""
    codes, scales = [], []
    for a in range(0, len(x), BLOCK):
        c, s = quantise_block(x[a:a + BLOCK], ts)
        codes += c
        scales.append(s)
    c = np.array(codes, dtype=np.uint8)
    return c[0::2] | (c[1::2] << 4), np.array(scales, dtype=np.uint8)


def values(codes, scales, ts: float):
    """Float64 values [..., D] of packed codes [..., D / 2] and scales."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    c = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],))
    c[..., 0::2] = E2M1[codes & 15]
    c[..., 1::2] = E2M1[codes >> 4]
    return c * np.repeat(E4M3[scales], BLOCK, axis=-1)[..., :c.shape[-1]] * ts


def attend(q, k, v, n: int, scale: float):
    """q [R, T, D] of the R query heads of one key/value head, k, v [cap, D], n slots
    in use; query i sees the slots j <= n - T + i. Returns (o, lse, weights [R, T, n])."""
    R, T, D = q.shape
    o, lse, w = np.zeros((R, T, D)), np.full((R, T), -np.inf), np.zeros((R, T, n))
    for i in range(T):
        m = n - T + i + 1
        if m <= 0:
            continue
        s = q[:, i] @ k[:m].T * scale
        top = s.max(-1, keepdims=True)
        e = np.exp(s - top)
        total = e.sum(-1, keepdims=True)
        w[:, i, :m] = e / total
        o[:, i] = w[:, i, :m] @ v[:m]
        lse[:, i] = (top + np.log(total))[:, 0]
    return o, lse, w


def key_mass(q, k, lse, chunks, scale: float):
    """q [R, T, D] and lse [R, T] of the query heads of one key/value head, k [T, D]:
    the weight of each key over the rows of the chunks."""
    R, T, _ = q.shape
    mass = np.zeros(T)
    for qb, qe, ctx, _ in chunks:
        for r in range(R):
            s = q[r, qb:qe] @ k[ctx:qe].T * scale
            seen = np.arange(ctx, qe)[None, :] <= np.arange(qb, qe)[:, None]
            with np.errstate(over="ignore", invalid="ignore"):
                w = np.where(seen & np.isfinite(lse[r, qb:qe])[:, None], np.exp(s - lse[r, qb:qe, None]), 0.0)
            mass[ctx:qe] += w.sum(0)
    return mass


def evict(mass, n: int, keep: int, recent: int):
    """The slots that stay, in order: the last min(recent, keep) of the n in use and
    those of the others with the highest mass; ties the lowest slot, NaN the highest."""
    m = min(n, keep)
    r = min(recent, m)
    key = [(0 if np.isnan(mass[j]) else 1, 0.0 if np.isnan(mass[j]) else -float(mass[j]), j) for j in range(n - r)]
    return sorted(j for _, _, j in sorted(key)[:m - r]) + list(range(n - r, n))
