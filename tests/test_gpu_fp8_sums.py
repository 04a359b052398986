"""The e4m3 products' sums are held in f32, for rows of every type.

The inputs here have products of 448 * 448 that cancel in pairs beside products
of 1/2 to 4, in every run of 8 positions: all products and partial sums are
multiples of 1/2 below 2^23, so f32 sums are exact in any order and only the
output's rounding is left, while sums of fewer bits lose the small products.
The bounds of ordinary inputs count f32 roundings and nothing else: a product
sums exact terms of 128 and ceil(K/128) block sums with two multiplications each,
(128 + K/128 + 4) 2^-24 of the sum of absolute values, then one rounding."""
import numpy as np
import pytest
import torch

from _block import DTYPES, U32, f64, gpu, normal, rounded, within
from _gpu import flush, setup
from oracle import fp8block

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def moe():
    return setup()


def _cancelling(gen, T, N, K):
    """(x [T, K], w [N, K]) as float32 e4m3 values; every block of x has absmax 448."""
    pick = lambda shape, values: torch.tensor(values)[torch.randint(len(values), shape, generator=gen)]  # noqa: E731
    x = pick((T, K // 8, 8), [-2.0, -1.0, 1.0, 2.0])
    w = pick((N, K // 8, 8), [-2.0, -1.0, -0.5, 0.5, 1.0, 2.0])
    a, b = (torch.randperm(8, generator=gen)[:2].tolist())
    x[:, :, a] = x[:, :, b] = 448.0
    w[:, :, a] = pick((N, K // 8), [256.0, 320.0, 416.0, 448.0])
    w[:, :, b] = -w[:, :, a]
    return x.reshape(T, K), w.reshape(N, K)


# streams and every tile shape, sizes that are no multiple of a tile
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,K", [(1, 264, 272), (16, 136, 1040), (5, 8200, 144), (33, 72, 400), (64, 1032, 272),
                                   (200, 1032, 144), (300, 4104, 272), (600, 4104, 144), (1100, 4104, 144),
                                   (2100, 4104, 144)])
def test_linear_keeps_small_products(moe, T, N, K, dtype):
    flush(f"fp8 sums T={T} N={N} K={K} {dtype}")
    x, w = _cancelling(torch.Generator().manual_seed(T + N), T, N, K)
    out = moe.moe_fp8_linear(moe.FP8Matrix(gpu(w.to(FP8)), torch.ones(-(-N // 128), -(-K // 128), device="cuda")),
                             gpu(x.to(dtype)))
    want = (x.double() @ w.double().t()).to(dtype)
    assert want.abs().max() > 4
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,K", [(1, 2048, 2048), (16, 264, 4112), (40, 520, 1040), (130, 392, 2064), (520, 1032, 400)])
def test_linear_within_the_bound_of_f32_sums(moe, T, N, K, dtype):
    flush(f"fp8 bound T={T} N={N} K={K} {dtype}")
    gen = torch.Generator().manual_seed(T + K)
    codes = (torch.randn(N, K, generator=gen) * 100).clamp(-448, 448).to(FP8)
    scales = (torch.rand(-(-N // 128), -(-K // 128), generator=gen) + 0.5) / 100
    x = normal(gen, (T, K), dtype)
    out = moe.moe_fp8_linear(moe.FP8Matrix(gpu(codes), gpu(scales)), gpu(x))
    ref, mag = fp8block.linear(x.float().numpy(), fp8block.matrix(codes.double().numpy(), scales.numpy()))
    within(out, ref, rounded(ref, dtype, (128 + -(-K // 128) + 4) * U32 * mag), "linear")


@pytest.mark.parametrize("T,E,K,H,I", [(4, 4, 2, 256, 128), (13, 8, 3, 384, 256), (40, 4, 2, 256, 128),
                                       (300, 4, 2, 128, 256)])
def test_experts_keep_small_products(moe, T, E, K, H, I):
    """gate and up are exact by the argument above, and down is the identity (or
    zero), so y is h = silu(g) u after its quantisation: half a step of e4m3
    (2^-4 of the value, 2^-10 of the scale below 2^-6 of it) and of bf16, and
    1e-5 for the f32 exponential."""
    flush(f"fp8 expert sums T={T} H={H} I={I}")
    gen = torch.Generator().manual_seed(T)
    x, gu = _cancelling(gen, T, E * 2 * I, H)
    dn = torch.zeros(E, H, I)
    n = min(H, I)
    dn[:, range(n), range(n)] = 1.0
    ones = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    gs = ones(E, 2 * I // 128, H // 128)
    gs[:, :I // 128] /= 32  # gates of a few units
    W = moe.FP8Weights(gpu(gu.to(FP8)).view(E, 2 * I, H), gs, gpu(dn.to(FP8)), ones(E, H // 128, I // 128), E, H, I, False)
    ids = torch.topk(torch.randn(T, E, generator=gen), K, dim=1).indices.int()
    _, offsets, sorted_slot, slot_pos, groups = moe.moe_permute(gpu(ids), E, False)
    y = f64(moe.moe_fp8_expert_ffn(W, gpu(x.bfloat16()), K, offsets, sorted_slot, groups))
    z = torch.einsum("th,enh->ten", x.double(), gu.view(E, 2 * I, H).double()).numpy()
    pos = slot_pos.cpu().numpy()
    worst = 0.0
    for t in range(T):
        for k in range(K):
            g, u = z[t, ids[t, k], :I] / 32, z[t, ids[t, k], I:]
            h = g / (1 + np.exp(-g)) * u
            a = np.repeat(np.abs(h).reshape(-1, 128).max(1), 128)
            step = np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * a / 448)
            bound = (step + 1e-5 * np.abs(h)) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(h) + 1e-30
            got = y[pos[t * K + k], :n]
            worst = max(worst, float((np.abs(got - h[:n]) / bound[:n]).max()))
    assert np.abs(z).max() > 4 and worst <= 1, worst
