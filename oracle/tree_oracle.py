"""Plain fp64 / integer restatement of rotary positions, 8-bit cache rows and trees
of drafted tokens.  One row or request at a time; shares no code with the kernels."""

from __future__ import annotations

import math

import numpy as np


def turns(position, freq):
    """Fraction of a turn in [0, 1), exact: freq counts 2^-64 turns a position."""
    return (int(position) * int(freq) % 2 ** 64) / 2.0 ** 64


def rope(x, positions, freqs, interleaved=False, amplitude=1.0):
    """x [n, heads, D]: the turned rows, and |x| + |y| of each pair, what roundings
    scale with (|x| itself behind the pairs)."""
    x = np.asarray(x, np.float64)
    n, half = x.shape[0], len(freqs)
    angle = 2 * math.pi * np.array([[turns(p, f) for f in freqs] for p in positions]).reshape(n, half)
    cos, sin = amplitude * np.cos(angle)[:, None], amplitude * np.sin(angle)[:, None]
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    out, mag = x.copy(), np.abs(x)
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(amplitude)
    return out, mag


def exponent(row):
    """The smallest e in [-100, 119] with the largest finite magnitude <= 448 * 2^e."""
    row = np.abs(np.asarray(row, np.float64))
    top = float(np.max(row[np.isfinite(row)], initial=0.0))
    e = -100
    while e < 119 and top > math.ldexp(448.0, e):
        e += 1
    return e


def e4m3(x):
    """x rounded to e4m3's numbers, ties to even; 448 at most; NaN for what is not finite."""
    x = np.asarray(x, np.float64)
    fine = np.isfinite(x)
    a = np.where(fine, np.abs(x), 0.0)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -60))), -6) - 3)
    y = np.minimum(np.round(a / step) * step, 448.0)  # numpy rounds ties to even
    return np.where(fine, np.copysign(y, x), np.nan)


def code_value(code):
    """An e4m3 code (0 .. 255) as a number."""
    s, e, m = code >> 7, code >> 3 & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    v = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
    return -v if s else v


def ancestors(parents):
    """{row: set of itself and all above it}; a parent out of range is none."""
    out = []
    for i, p in enumerate(parents):
        out.append({i} | (out[p] if 0 <= p < i else set()))
    return out


def accept(tokens, nxt, parents):
    """(path, tokens given out) of one request; a next token below 0 is none."""
    at, path = 0, [0]
    while True:
        kids = [c for c in range(at + 1, len(tokens)) if parents[c] == at and tokens[c] == nxt[at] >= 0]
        if not kids:
            return path, [nxt[i] for i in path]
        at = kids[0]
        path.append(at)


def attention(q, k, v, scale, seen):
    """q [l, Hq, D], k and v [n, Hk, D], seen [l, n]: out, lse and mag = sum p |v|."""
    l, Hq, D = q.shape
    Hk = k.shape[1]
    out, mag, lse = np.zeros((l, Hq, D)), np.zeros((l, Hq, D)), np.full((l, Hq), -np.inf)
    for j in range(l):
        t = np.flatnonzero(seen[j])
        if t.size == 0:
            continue
        for h in range(Hk):
            g = slice(h * Hq // Hk, (h + 1) * Hq // Hk)
            s = scale * (q[j, g] @ k[t, h].T)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(1, keepdims=True)
            out[j, g] = e @ v[t, h] / z
            mag[j, g] = e @ np.abs(v[t, h]) / z
            lse[j, g] = (m + np.log(z))[:, 0]
    return out, lse, mag
