"""The norms before and after a block with its gate and residual scale, and
their gradients, in fp64 (test infrastructure only).

  u = y rstd(y) w_post,  r = a res + b c u,  n = r rstd(r) w_pre

with rstd(v) = (mean(v^2) + eps)^-1/2 and c = 1 or sigmoid(gate) ([T] or [T, H]).

`magnitudes=True` evaluates the gradient's formula with every term's absolute
value, the scale of its f32 error.

Pins: the gradients against central differences of the forward functions.
"""
from __future__ import annotations

import numpy as np

from .router import sigmoid


def rstd_of(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1) + eps)


def _gate(gate, shape):
    if gate is None:
        return np.ones(shape)
    c = sigmoid(np.asarray(gate, dtype=np.float64))
    return np.broadcast_to(c[:, None] if c.ndim == 1 else c, shape)


def post(res, y, gate, w_post, a, b, eps):
    """(r, rstd of y or None, |b c u|): the residual stream after the block."""
    rstd = None
    u = y
    if w_post is not None:
        rstd = rstd_of(y, eps)
        u = y * rstd[:, None] * w_post
    u = b * _gate(gate, y.shape) * u
    return a * res + u, rstd, np.abs(u)


def pre(r, w_pre, eps):
    rstd = rstd_of(r, eps)
    return r * rstd[:, None] * w_pre, rstd


def grad(dr, dn, r, y, gate, w_post, w_pre, rstd_post, rstd_pre, a, b, magnitudes=False):
    """dict of dres, dy, dgate, dw_post, dw_pre from the given statistics."""
    m = np.abs if magnitudes else (lambda v: v)
    sign = 1.0 if magnitudes else -1.0
    out = {}
    D = m(dr) if dr is not None else np.zeros(r.shape)
    if w_pre is not None:
        s = rstd_pre[:, None]
        xh, g = m(r * s), m(dn * w_pre)
        D = D + s * (g + sign * xh * (g * xh).mean(axis=1, keepdims=True))
        out["dw_pre"] = (m(dn) * xh).sum(axis=0)
    if y is None:
        out["dres"] = D
        return out
    out["dres"] = abs(a) * D if magnitudes else a * D
    c = _gate(gate, y.shape)
    yh = m(y * rstd_post[:, None]) if w_post is not None else m(y)
    wp = m(w_post) if w_post is not None else np.ones(y.shape[1])
    bD = abs(b) * D if magnitudes else b * D
    if gate is not None:
        rest = _gate(-np.asarray(gate, dtype=np.float64), y.shape)  # 1 - c, without cancellation
        full = c * rest * bD * yh * wp
        out["dgate"] = full.sum(axis=1) if np.ndim(gate) == 1 else full
    du = bD * c
    if w_post is None:
        out["dy"] = du
        return out
    out["dw_post"] = (du * yh).sum(axis=0)
    g = du * wp
    out["dy"] = rstd_post[:, None] * (g + sign * yh * (g * yh).mean(axis=1, keepdims=True))
    return out
