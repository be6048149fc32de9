"""Plain fp64 restatement of the paged-cache and prompt operators (numpy, one
sequence and head at a time); shares no code with the library.

Arrays are float64 unless said otherwise.  ``attend`` also returns what error
bounds are made of: the sum of the weights times |v|, and the largest scale
times sum |q||k| of a row's scores.
"""
from __future__ import annotations

import math

import numpy as np

QMAX = {"int8": 127.0, "e4m3": 448.0}


def e4m3_value(code: int) -> float:
    """Value of an e4m3 code (sign, four exponent bits of bias 7, three mantissa bits)."""
    e, m = (code >> 3) & 15, code & 7
    v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if code & 128 else v


def quantise(x, kind):
    """Codes (int64: the number for int8, the byte for e4m3) and the fp32 scale
    of one row of exact values."""
    from fractions import Fraction as F
    x = [float(v) for v in x]
    n = len(x)
    if not all(math.isfinite(v) for v in x):
        return np.zeros(n, np.int64), np.float32(np.nan)
    top = max(abs(v) for v in x)
    if top < 2.0 ** -100:
        return np.zeros(n, np.int64), np.float32(0)
    scale = np.float32(top) / np.float32(QMAX[kind])
    s = F(float(scale))
    codes = []
    grid = [F(e4m3_value(c)) for c in range(127)]
    for v in x:
        y = abs(F(v)) / s
        if kind == "int8":
            c = int(y)
            if y - c > F(1, 2) or (y - c == F(1, 2) and c % 2):
                c += 1
            c = min(c, 127)
            codes.append(-c if v < 0 else c)
        else:
            lo = max(i for i in range(127) if grid[i] <= y)
            c = lo
            if lo < 126:
                mid = (grid[lo] + grid[lo + 1]) / 2
                if y > mid or (y == mid and lo % 2):
                    c = lo + 1
            codes.append(c | (128 if math.copysign(1, v) < 0 else 0))
    return np.array(codes, np.int64), scale


def value(codes, scale, kind):
    """Values a row's codes stand for."""
    c = codes.astype(np.float64) if kind == "int8" else np.array(
        [e4m3_value(int(b)) for b in np.asarray(codes).reshape(-1)]).reshape(np.shape(codes))
    return c * np.float64(scale)


def attend(q, k, v, scale):
    """q [nq, hq, d], the last nq positions of k, v [nk, hkv, d]: out [nq, hq, d],
    lse [nq, hq], weight [nq, hq, d] = sum p |v|, reach [nq, hq]."""
    nq, hq, d = q.shape
    nk, hkv, _ = k.shape
    out, wt = np.zeros((nq, hq, d)), np.zeros((nq, hq, d))
    lse, reach = np.full((nq, hq), -np.inf), np.zeros((nq, hq))
    for u in range(nq):
        seen = nk - nq + u + 1
        if seen <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:seen, h // (hq // hkv)], v[:seen, h // (hq // hkv)]
            with np.errstate(invalid="ignore", over="ignore"):
                s = kk @ q[u, h] * scale
                m = s.max()
                p = np.exp(s - m) if np.isfinite(m) else np.full(seen, np.nan)
                z = p.sum()
                out[u, h] = p @ vv / z
                wt[u, h] = p @ np.abs(vv) / z
                lse[u, h] = m + np.log(z) if np.isfinite(m) else m
                reach[u, h] = (np.abs(kk) @ np.abs(q[u, h])).max() * scale
    return out, lse, wt, reach
