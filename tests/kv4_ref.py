"""Plain 64-bit definitions of the attention-side operators (include/q8kv4.h),
on the CPU, for the tests: rotary positions, the 4-bit block, attention."""

from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rotate(x, pos, freq, interleaved=False, amplitude=1.0):
    """x [rows, heads, dim], float64 result; the first 2 * len(freq) values of
    a head turn by pos * freq."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(freq, dtype=np.float64)
    n = f.size
    th = np.asarray(pos, dtype=np.float64)[:, None, None] * f
    c, s = amplitude * np.cos(th), amplitude * np.sin(th)
    y = x.copy()
    ia, ib = ((np.arange(n) * 2, np.arange(n) * 2 + 1) if interleaved
              else (np.arange(n), np.arange(n) + n))
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    return y


def hold(x):
    """What the cache holds of fp32 values x [..., dim]: float64, NaN for the
    blocks with a NaN or an infinity."""
    x = np.asarray(x, dtype=np.float32)
    b = x.astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    out = np.empty_like(b)
    flat_in, flat_out = b.reshape(-1, 32), out.reshape(-1, 32)
    a = np.abs(flat_in).max(-1)
    bad = ~np.isfinite(flat_in).all(-1)
    m, e = np.frexp(np.where(bad | (a == 0), 1.0, a))   # a = m 2^e, m in [.5, 1)
    e = e - 1 - 2
    e = np.where(a > 7 * np.ldexp(1.0, e), e + 1, e)
    e = np.where(a == 0, -125, np.clip(e, -125, 125))
    unit = np.ldexp(1.0, e)[:, None]
    y = np.minimum(np.abs(np.where(bad[:, None], 0.0, flat_in)) / unit, 6.0)
    dist = np.abs(y[..., None] - GRID)
    # nearest, the even index of two equally near
    best = dist.min(-1, keepdims=True)
    cand = dist == best
    first = cand.argmax(-1)
    last = 7 - cand[..., ::-1].argmax(-1)
    pick = np.where(first % 2 == 0, first, last)
    flat_out[:] = np.copysign(GRID[pick], flat_in) * unit
    flat_out[bad] = np.nan
    return out.reshape(x.shape)


def attend(q, k, v, pos, scale, window=0):
    """One sequence and one key/value head: q [rows, dim], k and v [positions,
    dim], pos [rows].  Returns (O, tolerance) in float64.

    The tolerance counts the fp32 roundings of an evaluation whose products
    are exact: a score is a sum of D terms (each entering as three exact
    pieces, so 3 D additions), an exponent carries the score's error, and the
    outputs are sums over L weighted values.  A sum of n terms of total
    magnitude M errs by about sqrt(n) 2^-24 M, four times which is allowed,
    and 16 single roundings (2^-24 each) for scaling, exponentials, the joins
    and the division."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    O = np.zeros((q.shape[0], v.shape[1]))
    tol = np.zeros_like(O)
    for r, p in enumerate(pos):
        if p < 0:
            continue
        lo = max(0, p + 1 - window) if window else 0
        kk, vv = k[lo:p + 1], v[lo:p + 1]
        s = scale * (kk @ q[r])
        mag = scale * (np.abs(kk) @ np.abs(q[r]))
        w = np.exp(s - s.max())
        w /= w.sum()
        O[r] = w @ vv
        n = p + 1 - lo
        e_s = 4 * np.sqrt(3 * q.shape[1]) * mag + 4 * np.abs(s) + 4 * np.abs(s.max())
        e_w = e_s + w @ e_s          # a weight's error and that of the sum it is divided by
        tol[r] = 2.0 ** -24 * ((w * (e_w + 4 * np.sqrt(n) + 16)) @ np.abs(vv)) + 1e-37
    return O, tol
