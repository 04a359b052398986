"""The dense block and its gradients where the gates are far from zero: on both sides, in
each output, relative to the value itself.

Rows that are unit vectors and weights that are unit matrices leave each output one term, so
that y shows h, dw_gu and dx show dg and du one by one.

Bounds.  e = exp(-g) in f32: its argument g log2(e) is off by |g| 2^-24 relative to the
result, the exponential, the sum, the reciprocal and the products by a unit each: s and 1 - s
by (2 |g| + 8) 2^-23 relative.  dg = dh u (s + g s (1 - s)) adds two terms, so its error is
that of the absolute values' sum.  s below f32's normal numbers (2^-126, from g = -87.3 on)
may be taken as zero: |g| s, and with it each of these factors, is below 89 x 2^-126 < 2^-119
there."""
import numpy as np
import pytest
import torch

from _block import SMALL, UNIT, f64, gpu, rounded, within
from _gpu import flush, setup
from oracle import dense

pytestmark = pytest.mark.gpu

GATES = [-200.0, -100.0, -90.0, -88.5, -87.5, -87.0, -85.0, -80.0, -76.0, -75.0, -74.0, -73.0, -72.0, -71.0, -70.0,
         -69.0, -60.0, -40.0, -20.0, -10.0, -5.0, -1.28, -1.0, 0.0, 1.0, 5.0, 20.0, 60.0, 87.0, 90.0, 200.0]
TINY = 2.0 ** -119  # of the factors of dh u, dh and u


@pytest.fixture(scope="module")
def moe():
    return setup()


def _gates(dtype):
    return GATES + ([-60000.0] if dtype == torch.float16 else [-1e30, 1e30])


def _relative(g):
    return (2 * np.abs(g) + 8) * 2.0 ** -23


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [5, 64, 200])
@pytest.mark.parametrize("up", [False, True])
def test_gradients(moe, dtype, T, up):
    """dx = [dg du] W with W the unit matrix for the gates, or for the up rows."""
    flush(f"far gates, gradients T={T} {dtype} up={up}")
    H = I = 64
    gen = torch.Generator().manual_seed(T)
    unit = torch.eye(H)
    rows = torch.randperm(max(T, H), generator=gen)[:T] % H
    x = unit[rows].to(dtype)
    dy = (unit[torch.randint(H, (T,), generator=gen)] * 4).to(dtype)
    Wd = (torch.randint(0, 2, (H, I), generator=gen) * 32.0 - 16).to(dtype)      # dh = +-64
    W = torch.cat([unit * (not up), unit * up]).to(dtype)
    g = torch.tensor(_gates(dtype))[torch.randint(len(_gates(dtype)), (T, I), generator=gen)]
    u = torch.randint(0, 2, (T, I), generator=gen) * 24.0 - 12
    gu = torch.cat([g, u], 1).to(dtype)
    dx, dw_gu, dw_dn = moe.moe_dense_ffn_grad(moe.DenseWeights(gpu(W), gpu(Wd)), gpu(dy), gpu(x), gpu(gu))
    g, u = f64(gu)[:, :I], f64(gu)[:, I:]
    with np.errstate(over="ignore"):
        ref = dense.grad(f64(dy), f64(x), g, u, f64(W), f64(Wd))
        s, rest = dense.sigmoid(g), dense.sigmoid(-g)
    dh = np.abs(ref["dh"])
    err = np.concatenate([dh * np.abs(u) * (s * (1 + np.abs(g) * rest) * _relative(g) + TINY),
                          dh * (np.abs(g) * s * _relative(g) + TINY)], 1)
    # rounded as an operand, then (a single term, exact) as an output: the same value again
    err = err + UNIT[dtype] * (np.abs(ref["dgu"]) + err) + SMALL[dtype]
    within(dx, ref["dx"], err[:, I:] if up else err[:, :I], "dx")
    # the sums over the rows of the same unit vector
    terms, bound = np.abs(ref["dgu"]).T @ f64(x), err.T @ f64(x)
    within(dw_gu, ref["dw_gu"], rounded(ref["dw_gu"], dtype, bound + T * 2.0 ** -24 * (terms + bound)), "dw_gu")
    h = np.abs(ref["h"])
    bound = np.abs(u) * TINY + _relative(g) * h
    bound = np.abs(f64(dy)).T @ (bound + UNIT[dtype] * (h + bound) + SMALL[dtype])
    bound = bound + T * 2.0 ** -24 * (np.abs(f64(dy)).T @ h + bound)
    within(dw_dn, ref["dw_dn"], rounded(ref["dw_dn"], dtype, bound), "dw_dn")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [1, 8, 16, 64, 200])
@pytest.mark.parametrize("keep", [False, True])
def test_forward(moe, dtype, T, keep):
    """Projections that are a column of the weights each; y = h."""
    flush(f"far gates, forward T={T} {dtype} keep={keep}")
    H = I = 64
    gen = torch.Generator().manual_seed(T)
    rows = torch.randperm(max(T, H), generator=gen)[:T] % H
    x, Wd = torch.eye(H)[rows].to(dtype), torch.eye(H).to(dtype)
    # h = g u stays inside f16 up to g = 200; the largest gates are negative there
    g = torch.tensor(_gates(dtype))[torch.randint(len(_gates(dtype)), (I, H), generator=gen)]
    u = torch.randint(0, 2, (I, H), generator=gen) * 24.0 - 12
    W = torch.cat([g, u]).to(dtype)
    got = moe.moe_dense_ffn(moe.DenseWeights(gpu(W), gpu(Wd)), gpu(x), keep=keep)
    y, kept = got if keep else (got, None)
    g, u = (f64(W)[:I].T)[rows.numpy()], (f64(W)[I:].T)[rows.numpy()]
    if keep:
        assert torch.equal(kept.cpu(), W.t()[rows].contiguous())
    with np.errstate(over="ignore"):
        h = dense.activate(g, u)
    within(y, h, rounded(h, dtype, _relative(g) * np.abs(h) + np.abs(u) * TINY), "y")
