"""Pins of the dense block's, the 8-bit integer products' and the gradient norm's oracles."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import dense, grad_norm, int8


def test_block_by_hand():
    # one value each way: g = 2, u = 3, y = silu(2) 3 5
    y = dense.forward(np.array([[1.0]]), np.array([[2.0], [3.0]]), np.array([[5.0]]))
    assert abs(y[0, 0] - 2 / (1 + math.exp(-2)) * 15) < 1e-13


@pytest.mark.parametrize("T,H,I", [(1, 1, 1), (3, 4, 5)])
def test_block_gradients_against_differences(T, H, I):
    rng = np.random.default_rng(T)
    x, gu, dn = rng.normal(size=(T, H)), rng.normal(size=(2 * I, H)), rng.normal(size=(H, I))
    dy = rng.normal(size=(T, H))
    got = dense.grad(dy, x, *dense.project(x, gu), gu, dn)
    eps = 1e-6
    for name, v in (("dx", x), ("dw_gu", gu), ("dw_dn", dn)):
        for i in np.ndindex(*v.shape):
            keep = v[i]
            v[i] = keep + eps
            up = (dy * dense.forward(x, gu, dn)).sum()
            v[i] = keep - eps
            down = (dy * dense.forward(x, gu, dn)).sum()
            v[i] = keep
            assert abs((up - down) / (2 * eps) - got[name][i]) < 1e-6, (name, i)


def test_codes_are_the_nearest():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 32)).astype(np.float32)
    x[1] = np.arange(32) / 2 - 8  # quotients on middles: absmax 127/2 gives steps of 1/2
    x[1, 31] = 63.5
    x[2] = 0
    x[3] *= 1e-35  # below half a step of the smallest scale, 2^-100 / 127 = 6e-33
    q, s = int8.quant(x)
    for t in range(5):
        a = max(np.abs(x[t]).max(), np.float32(2.0 ** -100))
        m = np.float32(127) / np.float32(a)
        for k in range(32):
            v = Fraction(float(np.float32(x[t, k] * m)))
            best = min(range(-127, 128), key=lambda c: (abs(v - c), c % 2))
            assert q[t, k] == best
            assert abs(Fraction(float(x[t, k])) - q[t, k] * Fraction(float(s[t]))) <= Fraction(float(s[t])) * Fraction(51, 100)
    assert np.abs(q).max(axis=1).tolist() == [127, 127, 0, 0, 127]


def test_rows_that_are_not_finite():
    x = np.zeros((3, 16), np.float32)
    x[0, 3], x[1, 5], x[2, 2] = np.nan, np.inf, 1
    q, s = int8.quant(x)
    assert np.isnan(s[:2]).all() and np.isfinite(s[2]) and not q[:2].any()


def test_norm_and_factor():
    rng = np.random.default_rng(1)
    grads = [rng.normal(size=n).astype(np.float32) for n in (1, 7, 100)]
    exact = math.sqrt(math.fsum(float(v) ** 2 for g in grads for v in g))
    assert abs(grad_norm.norm(grads) - exact) <= 1e-14 * exact
    assert grad_norm.factor32(2.0, 4.0) == 1 and grad_norm.factor32(0.0, 0.0) == 0
    c = grad_norm.factor32(8.0, 2.0)
    assert abs(Fraction(float(c)) - Fraction(2) / (Fraction(8) + Fraction(1, 10 ** 6))) < Fraction(1, 2 ** 25)
    assert np.isnan(grad_norm.factor32(np.nan, 1.0)) and grad_norm.factor32(np.inf, 1.0) == 0
