"""Gradients of gates far from zero: c (1 - c) keeps its relative accuracy on both
sides.  c and 1 - c are each good to 6 2^-24 (the exponential's last place, one
addition, one division), so the bounds are those of ordinary gates with 8 2^-24
for the second factor, relative to the formula of absolute values."""
import numpy as np
import pytest
import torch

from _block import DTYPES, U32, f64, gpu, normal, permutation, rounded, within
from _gpu import flush, setup
from oracle import block_norm, sort

pytestmark = pytest.mark.gpu
GATES = [0.0, 4.0, -4.0, 12.0, -12.0, 16.0, -16.0, 17.5, 18.0, 30.0, -30.0, 60.0, -60.0]


@pytest.fixture(scope="module")
def moe():
    return setup()


@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_gate(moe, dtype):
    T, K, H = len(GATES), 3, 264
    flush(f"saturated gates, combine {dtype}")
    gen = torch.Generator().manual_seed(1)
    pos, gate = permutation(gen, T, K, True), torch.tensor(GATES)
    y, dout, w = normal(gen, (T * K + T, H), dtype), normal(gen, (T, H), dtype), torch.rand(T, K, generator=gen)
    _, _, dg = moe.moe_combine_grad(gpu(dout), gpu(y), gpu(w), gpu(pos), K, True, gate=gpu(gate))
    *_, ref, _, mag = sort.combine_grad(f64(dout), f64(y), f64(w), pos.numpy(), K, True, f64(gate),
                                        np.zeros((T * K + T, H)))
    assert (mag > 0).all()
    within(dg, ref, (H + 12 + 8) * U32 * mag, "dgate")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["token", "element"])
@pytest.mark.parametrize("H", [264, 2056])
def test_norm_gate(moe, kind, dtype, H):
    flush(f"saturated gates, norm {kind} H={H} {dtype}")
    T = len(GATES)
    gen = torch.Generator().manual_seed(2)
    res, y, dr, dn = (normal(gen, (T, H), dtype) for _ in range(4))
    gate = torch.tensor(GATES)
    if kind == "element":
        gate = gate[torch.randint(T, (T, H), generator=gen)].to(dtype)
    wo, wr = torch.randn(H, generator=gen), torch.randn(H, generator=gen)
    r, _, sp, sn = moe.moe_block_norm(gpu(res), gpu(y), gate=gpu(gate), w_post=gpu(wo), w_pre=gpu(wr))
    got = moe.moe_block_norm_grad(gpu(dr), gpu(dn), r, gpu(y), gate=gpu(gate), w_post=gpu(wo), w_pre=gpu(wr),
                                  rstd_post=sp, rstd_pre=sn)
    args = (f64(dr), f64(dn), f64(r), f64(y), f64(gate), f64(wo), f64(wr), f64(sp), f64(sn), 1.0, 1.0)
    ref, mag = block_norm.grad(*args)["dgate"], block_norm.grad(*args, magnitudes=True)["dgate"]
    err = (72 + 8) * U32 * mag
    within(got[2], ref, err if kind == "token" else rounded(ref, dtype, err), "dgate")
