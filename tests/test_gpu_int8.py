"""Products in 8-bit integers on the GPU against the oracle.

Without the gate every step is defined to the bit: codes, exact integer sums, two
multiplications and a rounding, so the outputs are compared exactly.  Gated: the oracle's z
(exact too) through silu in fp64; on the GPU silu is off by (2 |z| + 8) 2^-23 relative, its
product by one more rounding, and the output is rounded once."""
import numpy as np
import pytest
import torch

from _block import DTYPES, U32, f64, gpu, normal, rounded, within
from _gpu import flush, setup
from oracle import dense, int8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


def _matrix(gen, N, K):
    codes = torch.randint(-128, 128, (N, K), generator=gen, dtype=torch.int8)
    return codes, (torch.rand(N, generator=gen) + 0.5) / (64 * K ** 0.5)


def _z(x, codes, scales):
    return int8.linear32(x.float().numpy(), codes.numpy(), scales.numpy())


def _check(moe, x, codes, scales, gated, dtype):
    M = moe.Int8Matrix(gpu(codes), gpu(scales))
    out = moe.moe_int8_linear(M, gpu(x), gated=gated)
    N = len(scales)
    assert out.dtype == dtype and out.shape == (len(x), N // 2 if gated else N)
    z = _z(x, codes, scales)
    if not gated:
        want = torch.from_numpy(z).to(dtype)
        same = (out.cpu() == want) | (torch.isnan(out.cpu()) & torch.isnan(want))
        assert same.all(), f"{int((~same).sum())} of {same.numel()} differ"
    else:
        g, u = z[:, :N // 2].astype(np.float64), z[:, N // 2:].astype(np.float64)
        ref = dense.activate(g, u)
        within(out, ref, rounded(ref, dtype, ((2 * np.abs(g) + 8) * 2.0 ** -23 + U32) * np.abs(ref) + 2.0 ** -140), "gated")
    assert torch.equal(out.view(torch.uint8), moe.moe_int8_linear(M, gpu(x), gated=gated).view(torch.uint8))
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K", [(1, 16), (3, 128), (7, 144), (2, 2048), (130, 272), (5, 8208), (4, 65536), (1030, 64)])
def test_quant_is_bit_exact(moe, T, K, dtype):
    flush(f"int8 quant T={T} K={K} {dtype}")
    gen = torch.Generator().manual_seed(K)
    x = normal(gen, (T, K), dtype)
    x[0, 0] = 0.0
    x[T // 2] *= 2.0 ** -7
    x[T - 1, :16] = 0
    if dtype != torch.float16:
        x[0, 4], x[T - 1, 5] = 3e38, 1e-38
    q, s = moe.moe_int8_quant(gpu(x))
    rq, rs = int8.quant(x.float().numpy())
    assert q.dtype == torch.int8 and np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quant_ties_and_tiny_rows(moe):
    x = torch.zeros(4, 64)
    x[0] = torch.arange(64) / 2 - 16
    x[0, 63] = 63.5   # steps of 1/2: every other value lies on the middle of two codes
    x[1] = 2.0 ** -149
    x[2] = -2.0 ** -100
    q, s = moe.moe_int8_quant(gpu(x))
    rq, rs = int8.quant(x.numpy())
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    assert q[0, 30] == -2 and q[0, 31] == -1 and not q[1].any() and (q[2] == -127).all() and not q[3].any()


# one row, few rows, tile edges, K and N that end inside a step or tile
LINEAR = [(1, 8, 16), (1, 4096, 4096), (2, 264, 144), (4, 16, 65536), (8, 136, 1040), (15, 8200, 272), (16, 24, 4112),
          (17, 8, 16), (33, 128, 400), (64, 520, 256), (65, 72, 2064), (129, 136, 128), (200, 1032, 384), (257, 264, 112),
          (300, 392, 640), (513, 4168, 160), (90, 10248, 400)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(moe, T, N, K, dtype):
    flush(f"int8 linear T={T} N={N} K={K} {dtype}")
    gen = torch.Generator().manual_seed(T + N + K)
    codes, scales = _matrix(gen, N, K)
    _check(moe, normal(gen, (T, K), dtype), codes, scales, False, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,K", [(1, 16, 16), (1, 4096, 2048), (3, 272, 144), (16, 1040, 80), (17, 16, 2064),
                                   (65, 208, 400), (130, 528, 256), (300, 2064, 144), (2050, 4112, 48)])
def test_gated(moe, T, N, K, dtype):
    flush(f"int8 gated T={T} N={N} K={K} {dtype}")
    gen = torch.Generator().manual_seed(T + N + K)
    codes, scales = _matrix(gen, N, K)
    _check(moe, normal(gen, (T, K), dtype), codes, scales * 4, True, dtype)


@pytest.mark.parametrize("T,N,K", [(4100, 4104, 80), (2100, 8200, 144)])
def test_large_tiles(moe, T, N, K):
    flush(f"int8 large T={T} N={N} K={K}")
    gen = torch.Generator().manual_seed(T)
    codes, scales = _matrix(gen, N, K)
    _check(moe, normal(gen, (T, K), torch.bfloat16), codes, scales, False, torch.bfloat16)


@pytest.mark.parametrize("T", [2, 40])
def test_largest_sums(moe, T):
    """Every code at its end: the sums pass 2^30 and stay exact."""
    K, N = 65536, 16
    x = torch.ones(T, K)
    x[1] = -1
    codes = torch.full((N, K), 127, dtype=torch.int8)
    codes[1::2] = -128
    scales = torch.full((N,), 2.0 ** -20)
    _check(moe, x, codes, scales, False, torch.float32)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [3, 50])
def test_rows_that_are_not_finite(moe, T, gated):
    gen = torch.Generator().manual_seed(T)
    codes, scales = _matrix(gen, 48, 272)
    x = normal(gen, (T, 272), torch.bfloat16)
    b = x.clone()
    b[0, 271], b[T - 1, 0] = float("nan"), float("-inf")
    M = moe.Int8Matrix(gpu(codes), gpu(scales))
    y, yb = (moe.moe_int8_linear(M, gpu(v), gated=gated) for v in (x, b))
    assert torch.isnan(yb[[0, T - 1]]).all() and torch.equal(y[1:-1], yb[1:-1])
    assert not moe.moe_int8_quant(gpu(b))[0][[0, T - 1]].any()


def test_python_refusals(moe):
    x = torch.zeros(4, 64, device="cuda")
    M = moe.Int8Matrix(torch.zeros(24, 64, dtype=torch.int8, device="cuda"), torch.zeros(24, device="cuda"))
    with pytest.raises(ValueError, match="x must be"):
        moe.moe_int8_linear(M, x[:, :32].contiguous())
    with pytest.raises(ValueError, match="int8"):
        moe.moe_int8_linear(moe.Int8Matrix(M.codes.view(torch.uint8), M.scales), x)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_int8_linear(moe.Int8Matrix(M.codes, M.scales[:8]), x)
    with pytest.raises(ValueError, match="float32"):
        moe.moe_int8_quant(x.double())
    err = moe.ops._lib.MoeError
    with pytest.raises(err, match="gated: 16"):
        moe.moe_int8_linear(M, x, gated=True)
    with pytest.raises(err):  # an empty tensor has no address
        moe.moe_int8_linear(M, x[:0])
