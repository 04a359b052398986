"""Token sort, weighted combine and their gradients in fp64 (test infrastructure only).

Slots are s = t*K + k for the routed experts, then T*K + t for the shared one;
slot_pos[s] is the row of slot s in expert order.  A routed slot outside
[0, T*K), or a shared one outside [0, T*K + T), is skipped.

Every function also returns the sum of the absolute values of what it adds,
from which the tests derive their f32 error bounds.

Pins: the gradients against central differences of the forward functions.
"""
from __future__ import annotations

import numpy as np

from .router import sigmoid


def _slots(slot_pos, T, K, has_shared):
    """(token, position, k or K for the shared slot) of every slot not skipped."""
    out = []
    for t in range(T):
        for k in range(K):
            p = int(slot_pos[t * K + k])
            if 0 <= p < T * K:
                out.append((t, p, k))
        if has_shared:
            p = int(slot_pos[T * K + t])
            if 0 <= p < T * K + T:
                out.append((t, p, K))
    return out


def _weight(w, gate, t, k):
    if k < w.shape[1]:
        return float(w[t, k])
    return 1.0 if gate is None else float(sigmoid(np.float64(gate[t])))


def dispatch(x, slot_pos, K, has_shared, xs):
    """xs with the rows of x at the positions of their slots."""
    xs = np.array(xs)
    for t, p, _ in _slots(slot_pos, x.shape[0], K, has_shared):
        xs[p] = x[t]
    return xs


def slot_sum(y, w, slot_pos, K, has_shared, gate=None):
    """Weighted sum of each token's rows (w of ones: the gradient of dispatch)."""
    T, H = w.shape[0], y.shape[1]
    out, mag = np.zeros((T, H)), np.zeros((T, H))
    for t, p, k in _slots(slot_pos, T, K, has_shared):
        term = _weight(w, gate, t, k) * y[p]
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def combine_grad(dout, y, w, slot_pos, K, has_shared, gate, dy):
    """(dy, dw, dgate, sum |.| of dw, sum |.| of dgate); dy starts from `dy`."""
    T = dout.shape[0]
    dy = np.array(dy, dtype=np.float64)
    dw, mw = np.zeros((T, K)), np.zeros((T, K))
    dg, mg = np.zeros(T), np.zeros(T)
    for t, p, k in _slots(slot_pos, T, K, has_shared):
        c = _weight(w, gate, t, k)
        dy[p] = c * dout[t]
        if k < K:
            dw[t, k] = np.dot(dout[t], y[p])
            mw[t, k] = np.dot(np.abs(dout[t]), np.abs(y[p]))
        elif gate is not None:
            slope = c * float(sigmoid(-np.float64(gate[t])))  # c (1 - c), without cancellation
            dg[t] = slope * np.dot(dout[t], y[p])
            mg[t] = slope * np.dot(np.abs(dout[t]), np.abs(y[p]))
    return dy, dw, dg, mw, mg


def route_topk_grad(ids, w, dw, E):
    """(dlogits, error scale): the softmax gradient over the chosen experts."""
    T, K = ids.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        mean = np.dot(w[t], dw[t])
        size = np.dot(w[t], np.abs(dw[t]))
        for k in range(K):
            e = int(ids[t, k])
            if 0 <= e < E:
                out[t, e] += w[t, k] * (dw[t, k] - mean)
                mag[t, e] += w[t, k] * (np.abs(dw[t, k]) + size)
    return out, mag
