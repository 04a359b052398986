"""Products in e4m3 with a scale per block of 128, in fp64 (test infrastructure only).

Rows are quantised in blocks of 128 along K: a = max(absmax, 2^-100),
s = fp32(a / 448), m = fp32(448 / a), q = e4m3(fp32(x * m)); weights carry an
fp32 scale per block of 128 x 128.

Because codes are decided by roundings, a value computed with a small error may
get the neighbouring code.  quant_range gives the codes' values for the whole
interval of what a value may be, from which the expert FFN's error bound follows
without guessing how many codes differ.

Pins: the e4m3 decoding (see formats); the quantisation against a brute-force
search over all codes; closed forms of the products.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode

BLOCK = 128
TINY = np.float32(2.0 ** -100)
_VALUES = np.unique(e4m3_decode(np.arange(0x7F)))          # 0 .. 448, ascending
_MIDS = (_VALUES[1:] + _VALUES[:-1]) / 2


def e4m3_round(v):
    """Nearest e4m3 value of each |v| <= 464 (ties to the even code); NaN stays."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    i = np.searchsorted(_MIDS, a, side="left")             # a <= mids[i]
    i = np.minimum(i, len(_MIDS))
    at_tie = (i < len(_MIDS)) & (a == _MIDS[np.minimum(i, len(_MIDS) - 1)])
    i = np.where(at_tie & (i % 2 == 1), i + 1, i)          # the even code of the two
    r = np.copysign(_VALUES[i], v)
    return np.where(np.isnan(v), np.nan, r)


def _blocks(K):
    return [(b, min(b + BLOCK, K)) for b in range(0, K, BLOCK)]


def quant(x):
    """(values of the codes [T, K] float64, scales [T, ceil(K/128)] float32) of float32 rows."""
    x = np.asarray(x, dtype=np.float32)
    q = np.empty(x.shape)
    s = np.empty((x.shape[0], -(-x.shape[1] // BLOCK)), dtype=np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        for i, (lo, hi) in enumerate(_blocks(x.shape[1])):
            v = x[:, lo:hi]
            a = np.fmax.reduce(np.abs(v), axis=1)           # drops NaN
            a = np.fmax(a, TINY).astype(np.float32)
            m = np.float32(448.0) / a
            s[:, i] = a / np.float32(448.0)
            q[:, lo:hi] = e4m3_round((v * m[:, None]).astype(np.float32))
    return q, s


def dequant_rows(q, s):
    return q * np.repeat(s.astype(np.float64), BLOCK, axis=1)[:, :q.shape[1]]


def matrix(values, scales):
    """W in fp64 from the codes' values [N, K] and the block scales."""
    N, K = values.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]
    return values * s


def cut(qx, sx, values, scales, cols=None):
    """Bound of what an f8 matrix instruction would cut off: it aligns each run
    of 8 products to the run's largest exponent E (a subnormal or zero factor
    counted as 2^-6 at most) and drops what lies below 2^(E - 13).  A product has 8
    significant bits, so only one below 2^(E - 6) loses any, less than 2^(E - 13)
    or all of itself.  cols: the weight rows that `values` are.  The kernels' sums
    cut nothing: a bound that adds this allows more than they need."""
    cols = np.arange(values.shape[0]) if cols is None else np.asarray(cols)
    def expo(v):
        with np.errstate(divide="ignore"):
            return np.maximum(np.floor(np.log2(np.abs(v))), -6)

    ex, ew = expo(qx), expo(values)
    total = np.zeros((qx.shape[0], values.shape[0]))
    for k in range(0, qx.shape[1], 8):
        p = np.abs(qx[:, None, k:k + 8] * values[None, :, k:k + 8])
        unit = np.exp2((ex[:, None, k:k + 8] + ew[None, :, k:k + 8]).max(axis=2, keepdims=True))
        lost = np.where(p < unit * 2.0 ** -6, np.minimum(p, unit * 2.0 ** -13), 0.0).sum(axis=2)
        s = sx[:, k // BLOCK].astype(np.float64)[:, None]
        total += lost * s * scales[cols // BLOCK, k // BLOCK].astype(np.float64)[None, :]
    return total


def linear(x, W):
    """(z, sum of |terms|) of float32 rows times W^T."""
    d = dequant_rows(*quant(x))
    return d @ W.T, np.abs(d) @ np.abs(W).T


def quant_range(h, err):
    """Dequantised values of h [R, K] (fp64) and, element by element, how far
    the value that a computation with |error| <= err gets may lie from it."""
    R, K = h.shape
    mid, off = np.empty((R, K)), np.empty((R, K))
    for lo, hi in _blocks(K):
        v, e = h[:, lo:hi], err[:, lo:hi]
        a = np.fmax(np.abs(v).max(axis=1), TINY)[:, None]
        # the block's absmax is off by at most the error of the elements that can be it
        da = np.where(np.abs(v) + e >= a - e.max(axis=1, keepdims=True), e, 0).max(axis=1, keepdims=True)
        eps = 2.0 ** -22                                    # the roundings of a, m and v * m
        q = e4m3_round(np.clip(v / a * 448, -448, 448))
        d = (e / a + np.abs(v) / a * (da / a + eps)) * 448
        t = np.clip(v / a * 448, -448, 448)
        up, dn = e4m3_round(np.clip(t + d, -448, 448)), e4m3_round(np.clip(t - d, -448, 448))
        mid[:, lo:hi] = q * a / 448
        off[:, lo:hi] = (np.maximum(np.abs(up - q), np.abs(dn - q)) * a / 448 * (1 + da / a)
                         + np.abs(q) * a / 448 * (da / a + eps))
    return mid, off


def expert(x, gu, dn, I):
    """(y, error bound before the final rounding) of one expert's rows: x float32
    [R, H]; gu ([2I, H]) and dn ([H, I]): pairs of the codes' values and scales."""
    H = x.shape[1]
    z, mag = linear(x, matrix(*gu))
    ez = (BLOCK + H // BLOCK + 4) * 2.0 ** -24 * mag
    dnw = np.abs(matrix(*dn)).T
    g, u = z[:, :I], z[:, I:]
    sg = 1 / (1 + np.exp(-np.clip(g, -700, 700)))
    h = g * sg * u
    # |silu'| <= 1.1; the hardware's exponential and reciprocal are good to a
    # few units in the last place of 2^-23, the exponent's argument adds |g| units
    es = 1.1 * ez[:, :I] + np.abs(g * sg) * (8 + np.abs(g)) * 2.0 ** -23
    eh = es * (np.abs(u) + ez[:, I:]) + np.abs(g * sg) * ez[:, I:] + np.abs(h) * 2.0 ** -23
    hd, off = quant_range(h, eh)
    y = hd @ matrix(*dn).T
    bound = off @ dnw + (BLOCK + I // BLOCK + 4) * 2.0 ** -24 * ((np.abs(hd) + off) @ dnw)
    return y, bound
