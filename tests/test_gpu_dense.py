"""The dense gated feed-forward block and its gradients on the GPU against the fp64 oracle.

Bounds.  With U half a step of the rows' type, a sum over n products in f32 is off by
at most n 2^-24 of the sum of absolute values.  silu in f32: its exponential's argument
is off by |g| 2^-23, and six more operations round: (2 |g| + 8) 2^-23 relative; its slope
is at most 1.1.  h, dg and du, rounded once each as operands, add U of each value; each
output one more rounding.  Element by element these add up as absolute values (bound
`within`).  Against a fault that such a bound hides in a long sum stands a second one, on
the root mean square: independent roundings have at most U / sqrt(3) each, two of them
(the operand's and the output's) sqrt(2 / 3) U = 0.82 U of the output's, so U is the
limit wherever there are values enough (512) for that mean."""
import numpy as np
import pytest
import torch

from _block import SMALL, U32, UNIT, f64, gpu, normal, rounded, within
from _gpu import flush, setup
from oracle import dense

pytestmark = pytest.mark.gpu

HALVES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def moe():
    return setup()


def _make(gen, T, H, I, dtype):
    return (normal(gen, (T, H), dtype), normal(gen, (2 * I, H), dtype, H ** -0.5),
            normal(gen, (H, I), dtype, I ** -0.5))


def _rms(got, ref, dtype, name):
    err = f64(got) - ref
    if ref.size >= 512:
        rel = np.sqrt((err ** 2).mean() / (ref ** 2).mean())
        assert rel <= UNIT[dtype], f"{name}: rms error {rel / UNIT[dtype]:.3g} U"


def _silu_err(g):
    return (2 * np.abs(g) + 8) * 2.0 ** -23


def _check_forward(y, gu, x, W, Wd, dtype):
    U, S = UNIT[dtype], SMALL[dtype]
    x, W, Wd = f64(x), f64(W), f64(Wd)
    I, H = Wd.shape[1], Wd.shape[0]
    g, u = dense.project(x, W)
    mag = np.abs(x) @ np.abs(W).T * (H * U32)
    eg, eu = mag[:, :I], mag[:, I:]
    if gu is not None:
        within(gu, np.concatenate([g, u], 1), rounded(np.concatenate([g, u], 1), dtype, mag), "gu")
        _rms(gu, np.concatenate([g, u], 1), dtype, "gu")
    h = dense.activate(g, u)
    eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(g) * eu + _silu_err(g) * np.abs(h)
    eh = eh + U * (np.abs(h) + eh) + S
    err = eh @ np.abs(Wd).T + I * U32 * (np.abs(h) + eh) @ np.abs(Wd).T
    ref = h @ Wd.T
    within(y, ref, rounded(ref, dtype, err), "y")
    _rms(y, ref, dtype, "y")


# one row, few, tile edges, sizes that end inside a step of 64, more rows than a tile
SIZES = [(1, 8, 8), (1, 2048, 512), (2, 72, 8), (3, 264, 72), (8, 1024, 1032), (16, 520, 264), (17, 64, 1032),
         (33, 136, 200), (65, 1032, 520), (127, 128, 256), (129, 520, 136), (256, 512, 264), (300, 2056, 1032),
         (1000, 512, 512)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,H,I", SIZES)
def test_forward(moe, T, H, I, dtype, keep):
    flush(f"dense T={T} H={H} I={I} {dtype} keep={keep}")
    gen = torch.Generator().manual_seed(T + H + I)
    x, W, Wd = _make(gen, T, H, I, dtype)
    weights = moe.DenseWeights(gpu(W), gpu(Wd))
    got = moe.moe_dense_ffn(weights, gpu(x), keep=keep)
    y, gu = got if keep else (got, None)
    assert y.shape == (T, H) and y.dtype == dtype
    _check_forward(y, gu, x, W, Wd, dtype)
    again = moe.moe_dense_ffn(weights, gpu(x), keep=keep)
    assert torch.equal(y, again[0] if keep else again)


def _check_grad(got, dy, x, gu, W, Wd, dtype):
    U, S = UNIT[dtype], SMALL[dtype]
    dy, x, gu, W, Wd = (f64(v) for v in (dy, x, gu, W, Wd))
    T, (H, I) = len(x), Wd.shape
    g, u = gu[:, :I], gu[:, I:]
    ref = dense.grad(dy, x, g, u, W, Wd)
    a = np.abs
    edh = H * U32 * (a(dy) @ a(Wd))
    # the factors of dh in dg and du: |factor| and its own error
    fg, fu = dense.activate_grad(np.ones_like(g), g, u)
    edgu = np.concatenate([edh * a(fg) + (a(ref["dh"]) + edh) * (a(u) * 1.1 * _silu_err(g)),
                           edh * a(fu) + (a(ref["dh"]) + edh) * a(fu) * _silu_err(g)], 1)
    edgu = edgu + U * (a(ref["dgu"]) + edgu) + S
    m = a(ref["dgu"]) + edgu
    err = edgu @ a(W) + 2 * I * U32 * (m @ a(W))
    within(got[0], ref["dx"], rounded(ref["dx"], dtype, err), "dx")
    err = edgu.T @ a(x) + T * U32 * (m.T @ a(x))
    within(got[1], ref["dw_gu"], rounded(ref["dw_gu"], dtype, err), "dw_gu")
    eh = (_silu_err(g) + U) * a(ref["h"]) + S
    err = a(dy).T @ eh + T * U32 * (a(dy).T @ (a(ref["h"]) + eh))
    within(got[2], ref["dw_dn"], rounded(ref["dw_dn"], dtype, err), "dw_dn")
    for v, name in zip(got, ("dx", "dw_gu", "dw_dn")):
        _rms(v, ref[name], dtype, name)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,H,I", SIZES)
def test_gradients(moe, T, H, I, dtype):
    flush(f"dense gradients T={T} H={H} I={I} {dtype}")
    gen = torch.Generator().manual_seed(T + H + I + 1)
    x, W, Wd = _make(gen, T, H, I, dtype)
    gu, dy = normal(gen, (T, 2 * I), dtype), normal(gen, (T, H), dtype, 0.5)
    weights = moe.DenseWeights(gpu(W), gpu(Wd))
    got = moe.moe_dense_ffn_grad(weights, gpu(dy), gpu(x), gpu(gu))
    assert [tuple(v.shape) for v in got] == [(T, H), (2 * I, H), (H, I)]
    _check_grad(got, dy, x, gu, W, Wd, dtype)
    again = moe.moe_dense_ffn_grad(weights, gpu(dy), gpu(x), gpu(gu))
    assert all(torch.equal(v, w) for v, w in zip(got, again))


# tiles of the largest shapes, in every product: many rows, columns and both
LARGE = [(4100, 72, 2056), (2056, 4104, 72), (520, 2048, 4104), (4090, 72, 2040)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,H,I", LARGE)
def test_large(moe, T, H, I, dtype):
    flush(f"dense large T={T} H={H} I={I} {dtype}")
    gen = torch.Generator().manual_seed(T)
    x, W, Wd = _make(gen, T, H, I, dtype)
    weights = moe.DenseWeights(gpu(W), gpu(Wd))
    y, gu = moe.moe_dense_ffn(weights, gpu(x), keep=True)
    _check_forward(y, gu, x, W, Wd, dtype)
    dy = normal(gen, (T, H), dtype, 0.5)
    got = moe.moe_dense_ffn_grad(weights, gpu(dy), gpu(x), gu)
    _check_grad(got, dy, x, gu, W, Wd, dtype)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,H,I", [(5, 72, 24), (100, 264, 136), (700, 1032, 520), (2048, 2048, 2048),
                                   (2100, 1032, 2056), (4090, 2056, 4096)])
def test_gradients_of_whole_numbers_are_exact(moe, T, H, I, dtype):
    """g = 32 makes silu the identity to the last bit (exp(-32) < 2^-46): with sparse signs
    and small whole numbers every operand and sum is exact, so that one lost or repeated
    term, wherever it stands, shows."""
    gen = torch.Generator().manual_seed(I)

    def signs(shape, each):
        v = torch.randint(-1, 2, shape, generator=gen) * (torch.rand(shape, generator=gen) < each)
        return v.to(dtype)

    x, W = signs((T, H), 0.5), signs((2 * I, H), 0.5)
    dy = torch.zeros(T, H).to(dtype)   # one or two places a row: |dh| <= 2
    dy[torch.arange(T), torch.randint(0, H, (T,), generator=gen)] = 1
    dy[torch.arange(T), torch.randint(0, H, (T,), generator=gen)] = -1
    Wd = signs((H, I), 0.7)
    gu = torch.cat([torch.full((T, I), 32.0), torch.randint(-2, 3, (T, I), generator=gen).float()], 1).to(dtype)
    got = moe.moe_dense_ffn_grad(moe.DenseWeights(gpu(W), gpu(Wd)), gpu(dy), gpu(x), gpu(gu))
    dh = gpu(dy).double() @ gpu(Wd).double()
    u = gpu(gu[:, I:]).double()
    dgu = torch.cat([dh * u, dh * 32], 1)
    want = (dgu @ gpu(W).double(), dgu.t() @ gpu(x).double(), gpu(dy).double().t() @ (32 * u))
    assert max(float(v.abs().max()) for v in want) < 2 ** 24
    for a, b, name in zip(got, want, ("dx", "dw_gu", "dw_dn")):
        assert torch.equal(a, b.float().to(dtype)), name


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,H,I", [(3, 72, 24), (300, 264, 136)])
def test_rows_that_are_not_finite(moe, T, H, I, dtype):
    """NaN and infinities reach their own row's outputs only, also where they stand at the
    end of a row, behind which the next row's step ends."""
    gen = torch.Generator().manual_seed(T)
    x, W, Wd = _make(gen, T, H, I, dtype)
    dy, gu = normal(gen, (T, H), dtype), normal(gen, (T, 2 * I), dtype)
    weights = moe.DenseWeights(gpu(W), gpu(Wd))
    bad = [0, T // 2, T - 1] if T > 3 else [1]
    ok = [t for t in range(T) if t not in bad]
    xb, dyb = x.clone(), dy.clone()
    for i, t in enumerate(bad):
        xb[t, [0, H - 1, H // 2][i]] = [float("nan"), float("inf"), float("-inf")][i]
        dyb[t, [H - 1, 0, H // 2][i]] = [float("nan"), float("inf"), float("-inf")][i]
    y, yb = moe.moe_dense_ffn(weights, gpu(x)), moe.moe_dense_ffn(weights, gpu(xb))
    assert torch.isnan(yb[bad]).all() and torch.equal(y[ok], yb[ok])
    a = moe.moe_dense_ffn_grad(weights, gpu(dy), gpu(x), gpu(gu))
    b = moe.moe_dense_ffn_grad(weights, gpu(dyb), gpu(x), gpu(gu))
    assert not torch.isfinite(b[0][bad]).any() and torch.equal(a[0][ok], b[0][ok])


@pytest.mark.parametrize("dtype", HALVES)
def test_saturated_gates(moe, dtype):
    """Gates far out on both sides: silu's own limits, no NaN, no overflow on the way."""
    T, H, I = 40, 64, 72
    gen = torch.Generator().manual_seed(0)
    x, W, Wd = _make(gen, T, H, I, dtype)
    big = 60000.0 if dtype == torch.float16 else 1e30
    gu = normal(gen, (T, 2 * I), dtype)
    gu[:, :I] = torch.tensor([-big, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, big])[torch.randint(0, 8, (T, I), generator=gen)].to(dtype)
    gu[:, I:] *= 2.0 ** -4
    small = torch.where(gu[:, :I].abs() > 1000, torch.zeros(()), torch.ones(())).to(dtype)
    gu[:, I:] *= small  # where the gate itself is huge, h and dg would pass the type's range
    dy = normal(gen, (T, H), dtype, 2.0 ** -6)
    got = moe.moe_dense_ffn_grad(moe.DenseWeights(gpu(W), gpu(Wd)), gpu(dy), gpu(x), gpu(gu))
    I2 = f64(gu)[:, :I]
    assert torch.isfinite(got[2]).all()
    ref = dense.grad(f64(dy), f64(x), I2, f64(gu)[:, I:], f64(W), f64(Wd))
    err = f64(got[2]) - ref["dw_dn"]
    assert np.abs(err).max() <= 4 * UNIT[dtype] * np.abs(ref["dw_dn"]).max()


def test_given_outputs_and_workspaces(moe):
    """Outputs and workspaces of the caller are used, and rows behind them left alone."""
    T, H, I, dtype = 37, 136, 72, torch.bfloat16
    gen = torch.Generator().manual_seed(5)
    x, W, Wd = (gpu(v) for v in _make(gen, T, H, I, dtype))
    weights = moe.DenseWeights(W, Wd)
    y, gu = moe.moe_dense_ffn(weights, x, keep=True)

    def framed(*shape):
        n = int(np.prod(shape))
        f = torch.full((n + 256,), 7.0, dtype=dtype, device="cuda")
        return f, f[128:128 + n].view(*shape)

    fy, oy = framed(T, H)
    fg, og = framed(T, 2 * I)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    r = moe.moe_dense_ffn(weights, x, keep=True, ws=ws, out=oy, gu_out=og)
    assert r[0] is not None and torch.equal(oy, y) and torch.equal(og, gu)
    dy = gpu(normal(gen, (T, H), dtype))
    want = moe.moe_dense_ffn_grad(weights, dy, x, gu)
    frames = [framed(T, H), framed(2 * I, H), framed(H, I)]
    moe.moe_dense_ffn_grad(weights, dy, x, gu, ws=ws, dx=frames[0][1], dw_gu=frames[1][1], dw_dn=frames[2][1])
    for (f, o), w in zip(frames, want):
        assert torch.equal(o, w)
    for f in [fy, fg] + [f for f, _ in frames]:
        assert (f[:128] == 7).all() and (f[-128:] == 7).all()


def test_python_refusals(moe):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    W, Wd = torch.zeros(32, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(64, 16, dtype=torch.bfloat16, device="cuda")
    ok = moe.DenseWeights(W, Wd)
    for bad, text in ((moe.DenseWeights(W.float(), Wd.float()), "float16"), (moe.DenseWeights(W, Wd.half()), "bfloat16"),
                      (moe.DenseWeights(W[:31], Wd), "even"), (moe.DenseWeights(W, Wd.t()), "contiguous"),
                      (moe.DenseWeights(W, Wd[:32]), "shape")):
        with pytest.raises(ValueError, match=text):
            moe.moe_dense_ffn(bad, x)
    with pytest.raises(ValueError, match="bfloat16"):
        moe.moe_dense_ffn(ok, x.half())
    with pytest.raises(ValueError, match="shape"):
        moe.moe_dense_ffn(ok, x[:, :32].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_dense_ffn(ok, torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(ValueError, match="keep"):
        moe.moe_dense_ffn(ok, x, gu_out=torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_dense_ffn(ok, x, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        moe.moe_dense_ffn_grad(ok, x, x, x)
    err = moe.ops._lib.MoeError
    with pytest.raises(err):
        moe.moe_dense_ffn(ok, x[:0])
