"""Pins of the fp64 oracles of the token sort, the block norm and the e4m3
products: gradients against central differences, the quantisation against a
search over all codes, closed forms."""
import numpy as np
import pytest

from oracle import block_norm, fp8block, sort
from oracle.formats import e4m3_decode


def _perm(rng, T, K, has_shared):
    routed = rng.permutation(T * K)
    return np.concatenate([routed, T * K + rng.permutation(T)]) if has_shared else routed


def _diff(f, v, i, step=1e-6):
    a, b = v.copy(), v.copy()
    a[i] += step
    b[i] -= step
    return (f(a) - f(b)) / (2 * step)


@pytest.mark.parametrize("has_shared,gated", [(False, False), (True, False), (True, True)])
def test_combine_and_dispatch_gradients_against_differences(has_shared, gated):
    rng = np.random.default_rng(1)
    T, K, H = 5, 3, 8
    S = T * K + (T if has_shared else 0)
    pos = _perm(rng, T, K, has_shared)
    pos[4] = -1
    y, w = rng.standard_normal((S, H)), rng.random((T, K))
    gate = rng.standard_normal(T) if gated else None
    dout, cot = rng.standard_normal((T, H)), rng.standard_normal((S, H))
    dy, dw, dg, _, _ = sort.combine_grad(dout, y, w, pos, K, has_shared, gate, np.zeros((S, H)))
    f = lambda y, w, g: (sort.slot_sum(y, w, pos, K, has_shared, g)[0] * dout).sum()  # noqa: E731
    for i in [(0, 0), (7, 3), (S - 1, 7)]:
        assert abs(_diff(lambda v: f(v, w, gate), y, i) - dy[i]) < 1e-7
    for i in [(0, 0), (1, 1), (4, 2)]:
        assert abs(_diff(lambda v: f(y, v, gate), w, i) - dw[i]) < 1e-7
    if gated:
        assert abs(_diff(lambda v: f(y, w, v), gate, (2,)) - dg[2]) < 1e-7
    x = rng.standard_normal((T, H))
    dx, _ = sort.slot_sum(cot, np.ones((T, K)), pos, K, has_shared)
    d = lambda v: (sort.dispatch(v, pos, K, has_shared, np.zeros((S, H))) * cot).sum()  # noqa: E731
    for i in [(0, 0), (1, 5), (4, 7)]:
        assert abs(_diff(d, x, i) - dx[i]) < 1e-7


def test_topk_gradient_against_differences():
    rng = np.random.default_rng(2)
    T, E, K = 3, 9, 4
    z = rng.standard_normal((T, E))
    ids = np.argsort(-z, axis=1)[:, :K]
    dw = rng.standard_normal((T, K))

    def loss(z):
        p = np.exp(np.take_along_axis(z, ids, 1))
        return (p / p.sum(1, keepdims=True) * dw).sum()

    p = np.exp(np.take_along_axis(z, ids, 1))
    dz, _ = sort.route_topk_grad(ids, p / p.sum(1, keepdims=True), dw, E)
    for t in range(T):
        for e in range(E):
            assert abs(_diff(loss, z, (t, e)) - dz[t, e]) < 1e-8


@pytest.mark.parametrize("gate_kind", ["none", "token", "element"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_norm_gradients_against_differences(gate_kind, post, pre):
    rng = np.random.default_rng(3)
    T, H, a, b, eps = 3, 8, 0.7, -1.3, 1e-3
    v = dict(res=rng.standard_normal((T, H)), y=rng.standard_normal((T, H)))
    if gate_kind != "none":
        v["gate"] = rng.standard_normal(T if gate_kind == "token" else (T, H))
    if post:
        v["w_post"] = rng.standard_normal(H)
    if pre:
        v["w_pre"] = rng.standard_normal(H)
    dr, dn = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def loss(v):
        r, _, _ = block_norm.post(v["res"], v["y"], v.get("gate"), v.get("w_post"), a, b, eps)
        s = (r * dr).sum()
        return s + (block_norm.pre(r, v["w_pre"], eps)[0] * dn).sum() if pre else s

    r, rstd_post, _ = block_norm.post(v["res"], v["y"], v.get("gate"), v.get("w_post"), a, b, eps)
    rstd_pre = block_norm.rstd_of(r, eps)
    g = block_norm.grad(dr, dn, r, v["y"], v.get("gate"), v.get("w_post"), v.get("w_pre"), rstd_post,
                        rstd_pre, a, b)
    for name, key in (("res", "dres"), ("y", "dy"), ("gate", "dgate"), ("w_post", "dw_post"), ("w_pre", "dw_pre")):
        if name not in v:
            assert key not in g
            continue
        for i in np.ndindex(v[name].shape):
            num = _diff(lambda q: loss({**v, name: q}), v[name], i)
            assert abs(num - g[key][i]) < 2e-7 * (1 + abs(num)), (name, i)


def test_e4m3_rounding_is_the_nearest_value_with_ties_to_even():
    values = e4m3_decode(np.arange(0x7F))
    rng = np.random.default_rng(4)
    mids = (np.sort(values)[1:] + np.sort(values)[:-1]) / 2
    v = np.concatenate([rng.uniform(-448, 448, 2000), rng.uniform(-0.02, 0.02, 500), mids, -mids, values])
    got = fp8block.e4m3_round(v)
    for x, r in zip(v, got):
        d = np.abs(np.abs(x) - values)
        near = np.flatnonzero(d == d.min())
        want = values[near[near % 2 == 0][0]] if len(near) > 1 else values[near[0]]
        assert abs(r) == want and (r == 0 or np.sign(r) == np.sign(x))


def test_quantisation_of_special_blocks():
    x = np.zeros((4, 256), dtype=np.float32)
    x[1, 3], x[2, 130], x[3, 200] = 1e-38, np.nan, np.inf
    q, s = fp8block.quant(x)
    assert np.all(q[:2] == 0) and np.all(np.isfinite(s[:3]))
    assert np.isnan(q[2, 130]) and np.isnan(q[2]).sum() == 1
    assert np.isnan(q[3, 200]) and np.isinf(s[3, 1])


def test_products_of_representable_values_are_exact():
    rng = np.random.default_rng(5)
    x = rng.choice([-2.0, -1.0, 0.0, 1.0, 448.0], (3, 272)).astype(np.float32)
    x[:, ::128] = 448.0
    x[:, 256] = 448.0
    W = rng.choice([-1.0, 0.5, 2.0], (5, 272))
    z, _ = fp8block.linear(x, W)
    assert np.array_equal(z, x.astype(np.float64) @ W.T)


def test_quant_range_covers_every_value_of_the_interval():
    rng = np.random.default_rng(6)
    h = rng.standard_normal((6, 256))
    err = np.abs(h) * 1e-3 + 1e-4
    mid, off = fp8block.quant_range(h, err)
    for _ in range(50):
        v = (h + err * rng.uniform(-1, 1, h.shape)).astype(np.float32)
        d = fp8block.dequant_rows(*fp8block.quant(v))
        assert np.all(np.abs(d - mid) <= off + 1e-12)
