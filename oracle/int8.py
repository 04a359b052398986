"""Products in 8-bit integers with a scale per token and per channel (test
infrastructure only).

  a = max(absmax of the row, 2^-100), s = a / 127, q = rne(x (127 / a))
  z[t][n] = s[t] S[n] sum_k q[t][k] W[n][k]

The quantisation's three operations are fp32 by definition, the sums exact integers.

Pins: the codes against a search over all 255 of them in exact fractions, rows
whose quotients fall on the middle between two codes, and the error bound of half
a step.
"""
from __future__ import annotations

import numpy as np

FLOOR = np.float32(2.0 ** -100)


def quant(x):
    """(codes int64 [T, K], scales float32 [T]) of float32 rows; a row with a NaN or an
    infinity has codes 0 and scale NaN."""
    x = np.asarray(x, dtype=np.float32)
    a = np.abs(x).max(axis=1)
    bad = ~np.isfinite(a)
    a = np.where(bad, np.float32(1), np.maximum(a, FLOOR)).astype(np.float32)
    m = (np.float32(127) / a).astype(np.float32)
    v = np.where(bad[:, None], np.float32(0), x)
    q = np.rint((v * m[:, None]).astype(np.float32)).astype(np.int64)
    s = np.where(bad, np.float32(np.nan), (a / np.float32(127)).astype(np.float32))
    return q, s.astype(np.float32)


def sums(q, codes):
    """Exact integer sums [T, N]."""
    # below 2^53: exact in fp64
    return (q.astype(np.float64) @ codes.astype(np.float64).T).astype(np.int64)


def linear32(x, codes, scales):
    """z as the definition's own f32 steps give it: (f32(sum) * s) * S."""
    q, s = quant(x)
    z = sums(q, codes).astype(np.float32)
    return (z * s[:, None]).astype(np.float32) * np.asarray(scales, dtype=np.float32)[None, :]
