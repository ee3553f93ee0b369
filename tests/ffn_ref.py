"""The feed-forward side's operators in 64 bits, with numpy: what a microscaled
block holds, the products, the gated block and the norms, from their
definitions (include/q8ffn.h)."""

import math

import numpy as np

GRIDS = {
    "mx4": np.array([0, .5, 1, 1.5, 2, 3, 4, 6.]),
    "mx6": np.concatenate([np.arange(16) / 8, 2 + np.arange(8) / 4, 4 + np.arange(8) / 2]),
    "mx8": np.arange(128) / 64,
}
EMAX = {"mx4": 2, "mx6": 2, "mx8": 0}
BORDER = {"mx4": 7.0, "mx6": 7.75, "mx8": 127.5 / 64}
U = 2.0 ** -24  # half a step of fp32


def exponents(x, form):
    """Scale exponents of fp32 rows [..., K/32]; 128 for a block that is not finite."""
    b = np.abs(np.asarray(x, np.float32).astype(np.float64)).reshape(*x.shape[:-1], -1, 32)
    a = b.max(-1)
    bad = ~np.isfinite(b).all(-1)
    a = np.where(bad | (a == 0), 1.0, a)
    e = np.floor(np.log2(a)).astype(int)
    e = np.where(2.0 ** e > a, e - 1, np.where(2.0 ** (e + 1) <= a, e + 1, e)) - EMAX[form]
    e = np.clip(np.where(a > BORDER[form] * 2.0 ** e, e + 1, e), -120, 125)
    return np.where(bad, 128, e)


def codes(x, form):
    """(index of the magnitude, negative, scale exponent) of every value: the
    nearest magnitude, an even index on a tie."""
    e = exponents(x, form)
    g = GRIDS[form]
    y = np.asarray(x, np.float32).astype(np.float64).reshape(*x.shape[:-1], -1, 32)
    y = np.where((e == 128)[..., None], 0.0, y)
    y = np.minimum(np.abs(y) / 2.0 ** np.where(e == 128, 0, e)[..., None], g[-1])
    hi = np.clip(np.searchsorted(g, y), 1, len(g) - 1)
    up, down = g[hi] - y, y - g[hi - 1]
    i = np.where(up < down, hi, np.where(up > down, hi - 1, np.where(hi % 2 == 0, hi, hi - 1)))
    return i.reshape(x.shape), np.signbit(np.asarray(x, np.float32)), e


def hold(x, form):
    """What the blocks of fp32 rows hold, in 64 bits."""
    i, neg, e = codes(x, form)
    v = np.where(neg, -1.0, 1.0) * GRIDS[form][i]
    s = np.where(e == 128, np.nan, 2.0 ** np.where(e == 128, 0, e))
    return (v.reshape(*e.shape, 32) * s[..., None]).reshape(x.shape)


def mx4_bytes(idx, neg):
    """Packed codes uint8 [N][K/2] of magnitude indexes and signs."""
    n = (idx + 8 * neg).astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def mx4_values(codes_, scales):
    """The values of packed codes and scale bytes, 255 for NaN."""
    n = np.stack([codes_ & 15, codes_ >> 4], -1).reshape(*codes_.shape[:-1], -1)
    v = np.where(n & 8, -1.0, 1.0) * GRIDS["mx4"][n & 7]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(v.shape)


def product(w, x, pieces):
    """(sums [t][n], their error bound).  Products are exact; an instruction adds
    128 of them and the sum so far, with an error of at most 2^-23 of their
    magnitudes, ``pieces`` instructions to 128 columns; at most 16 waves' sums are
    added."""
    y = x @ w.T
    n = pieces * -(-w.shape[1] // 128) + 16
    return y, n * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


def activation(x, kind):
    with np.errstate(over="ignore"):
        if kind == "silu":
            return x / (1 + np.exp(-x))
        if kind == "gelu":
            return np.array([0.5 * v * math.erfc(-v / math.sqrt(2)) for v in x.ravel()]).reshape(x.shape)
        if kind == "gelu_tanh":
            return x / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
        return {"relu": lambda: np.maximum(x, 0), "sigmoid": lambda: 1 / (1 + np.exp(-x)), "identity": lambda: x}[kind]()


def gated(wg, wu, x, pieces, kind):
    """(h, its error bound): the sums' errors through the activation, whose slope
    is at most 1.13, and the activation's own arithmetic.  Its argument is rounded a
    few times, which an exponential of z turns into a relative error of |z| roundings;
    |z| is below 1.6 (|x| + 0.05 |x|^3) or x^2 / 2 + 1 here."""
    g, eg = product(wg, x, pieces)
    u, eu = product(wu, x, pieces)
    a = activation(g, kind)
    h = a * u
    z = {"gelu": g * g + 2, "gelu_tanh": 1.6 * (np.abs(g) + 0.05 * np.abs(g) ** 3)}.get(kind, np.abs(g))
    own = (16 + 8 * np.minimum(z, 700.0)) * U
    return h, 1.13 * eg * (np.abs(u) + eu) + np.abs(a) * eu + own * np.abs(h) + 2.0 ** -126 * (1 + np.abs(u))


def norm(x, kind, weight, bias, eps, offset):
    if kind is None:
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))
    if weight is not None:
        y = y * (weight.astype(np.float64) + float(np.float32(offset)))
    return y if bias is None else y + bias.astype(np.float64)
