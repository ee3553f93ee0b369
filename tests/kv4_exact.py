"""Attention inputs whose results depend on every bit of the queries and of
the softmax weights, with tolerances that count the roundings, and a model of
the kernel's number formats that can leave some of those bits out.

The kernel multiplies without error: a query value enters as six 6-bit pieces
(E2M3, each a power of two below the one before it: 2^-4, then 2^-5 four times)
and holds to 2^-29 of its block's largest value, a weight as three bf16 pieces,
all 24 bits.  A score is a sum of up to 6 ceil(D / 128) + 1 fp32 additions, an
output one of three for each 32 positions."""

from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative
PIECE_DOWN = (0, 4, 9, 14, 19, 24)


def _e2m3(x):
    """Nearest of the E2M3 numbers (steps 1/8 below 2, 1/4 below 4, 1/2 up to
    7.5), ties to even."""
    a = np.abs(x)
    step = np.where(a < 2, 0.125, np.where(a < 4, 0.25, 0.5))
    return np.copysign(np.minimum(np.rint(a / step) * step, 7.5), x)


def cut_query(q, pieces=6):
    """q [..., D] as its first pieces hold it, block by block of 32."""
    b = np.asarray(q, dtype=np.float64).reshape(*np.shape(q)[:-1], -1, 32)
    top = np.abs(b).max(-1, keepdims=True)
    m, e = np.frexp(np.where(top == 0, 1.0, top))     # top = m 2^e, m in [.5, 1)
    e = e - 1 - 2 + (2 * m > 1.875)
    left, out = b.copy(), np.zeros_like(b)
    for down in PIECE_DOWN[:pieces]:
        unit = np.ldexp(1.0, e - down)
        p = _e2m3(left / unit) * unit
        out += p
        left -= p
    return out.reshape(np.shape(q))


def cut_weight(w, bits=24):
    """Positive weights rounded to fp32 and truncated to their upper bits."""
    m, e = np.frexp(np.asarray(w, dtype=np.float64).astype(np.float32).astype(np.float64))
    return np.ldexp(np.floor(np.ldexp(m, bits)), e - bits)


def model(q, k, v, scale, pieces=6, bits=24):
    """softmax(scale q k^T) v for rows q [n, D] that see all of k and v
    [positions, D], the queries cut to `pieces` pieces and the weights, where
    they multiply values, to `bits` bits; all else in 64 bits."""
    s = scale * (cut_query(q, pieces) @ np.asarray(k, dtype=np.float64).T)
    w = np.exp(s - s.max(-1, keepdims=True))
    return cut_weight(w, bits) @ np.asarray(v, dtype=np.float64) / w.sum(-1, keepdims=True)


# Two positions, with the query's head a row.  Both functions return (q [heads,
# D], k [2, D], v [2, D], scale, expected [heads, D], tolerance [heads, D]);
# keys and values are numbers that the 4-bit blocks hold exactly.

def piece_case(heads, dim):
    """Head h's score needs piece h % 6 of its query and no other.  Its
    block's largest value, which no key looks at, is 4 2^d with d the piece's
    distance from the first, so that value 5 of the block, 0.875, is what that
    piece alone holds: over the scales of the pieces before it it is below
    1/16, half of their least step.  Scores 1 and 0, values v and -v:
    O = v tanh(1/2).

    In units of U: the weight of the second position takes 2 from its
    exponent (the scale and the product, each 1, times 1/e's exponent, 1) and 2
    from the exponential (one step); O moves by 0.4 of that.  The sum of two
    positions takes at most 8 |v| / (1 + 1/e), the sum of weights 1, its
    reciprocal 1 and the product 1: less than 16."""
    q = np.zeros((heads, dim), np.float32)
    for h in range(heads):
        q[h, 0] = 4.0 * 2.0 ** PIECE_DOWN[h % 6]
        q[h, 5] = 0.875
    k, v = np.zeros((2, dim), np.float32), np.zeros((2, dim), np.float32)
    k[0, 5] = 4.0
    v[0] = np.resize([6, -4, 3, 2, -1.5, 1, 0.5, -6], dim)
    v[1] = -v[0]
    scale = 1 / 3.5
    want = np.repeat(v[:1].astype(np.float64) * np.tanh(0.5), heads, 0)
    return q, k, v, scale, want, np.repeat(16 * U * np.abs(v[:1]), heads, 0)


def weight_case(heads, dim, seed=0):
    """Scores 0 and -x_h with x_h in 0.1 .. 3, values 0 and 6: O = 6 w / (1 + w)
    with w = e^-x_h, whose relative error is no smaller than half that of w.

    In units of U: 2 x_h from w's exponent (as above), 2 from the exponential,
    at most 8 from the sum, 3 from the sum of weights, its reciprocal and the product,
    and x_h / 32 from the query's 2^-29: less than 16 + 3 x_h."""
    rng = np.random.default_rng(seed)
    x = rng.uniform(0.1, 3.0, heads).astype(np.float32)
    q = np.zeros((heads, dim), np.float32)
    q[:, 5] = -x
    k, v = np.zeros((2, dim), np.float32), np.zeros((2, dim), np.float32)
    k[1, 5] = 4.0
    v[1] = 6.0
    w = np.exp(-x.astype(np.float64))[:, None]
    want = np.repeat(6 * w / (1 + w), dim, 1)
    return q, k, v, 0.25, want, (16 + 3 * x[:, None]) * U * want


# Relative error of the outputs' norm on rows of standard normal queries, keys
# and values with scale D^-1/2, up to 1500 positions: scores of size 1, weights
# whose errors are independent.  In units of U, roots of sums of squares: a score's
# 13 additions 4 (of numbers up to a few), its exponent 5, the exponential 2; at
# most 12 steps of a wave with 3 additions each 6 and the joins 3: 10, of which 16 are allowed.
NORM = 16 * U
