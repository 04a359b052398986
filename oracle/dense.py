"""The dense gated feed-forward block and its gradients in fp64 (test
infrastructure only).

  g = x Wg^T, u = x Wu^T, h = silu(g) u, y = h Wd^T

Pins: the gradients against central differences of the forward function.
"""
from __future__ import annotations

import numpy as np

from .router import sigmoid


def project(x, gu):
    """(g, u) [T, I] each."""
    z = x @ gu.T
    half = gu.shape[0] // 2
    return z[:, :half], z[:, half:]


def activate(g, u):
    return g * sigmoid(g) * u


def forward(x, gu, dn):
    return activate(*project(x, gu)) @ dn.T


def activate_grad(dh, g, u):
    """(dg, du)."""
    s = sigmoid(g)
    return dh * u * s * (1.0 + g * sigmoid(-g)), dh * g * s


def grad(dy, x, g, u, gu, dn):
    """dict of dx, dw_gu, dw_dn (and the inner dh, dgu and h) from the kept projections."""
    dh = dy @ dn
    dgu = np.concatenate(activate_grad(dh, g, u), axis=1)
    h = activate(g, u)
    return {"dh": dh, "dgu": dgu, "h": h, "dx": dgu @ gu, "dw_gu": dgu.T @ x, "dw_dn": dy.T @ h}
