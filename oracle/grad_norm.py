"""The norm of many gradients together and their scaling (test infrastructure only).

  norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  g' = c g

Pins: math.fsum of exact squares; the factor against its definition in fractions.
"""
from __future__ import annotations

import numpy as np


def norm(grads):
    total = 0.0
    for g in grads:
        v = np.asarray(g, dtype=np.float64).reshape(-1)
        total += float(np.dot(v, v))
    return np.sqrt(total)


def factor32(norm32, max_norm):
    """c as the definition's f32 steps give it from the f32 norm."""
    one = np.float32(1)
    with np.errstate(all="ignore"):
        c = np.float32(max_norm) / (np.float32(norm32) + np.float32(1e-6))
    return one if c > one else np.float32(c)
