"""The dense block in every shape of its tiles and streams, forward (projections kept or
not) and backward, and its weight gradients over more rows than 2^31 elements hold: on whole
numbers, where every sum is exact and one lost or repeated term shows.

test_tile_choice.py holds that FORWARD and GRADIENTS below take all the shapes."""
import pytest
import torch

import test_gpu_dense as base
from _block import gpu
from _gpu import flush, setup

pytestmark = pytest.mark.gpu

# (T, H, I); up to 16 rows stream: tiles of 8 rows and of 16, K below and from 4096 on
FORWARD = [(1, 72, 136), (5, 2056, 4104), (8, 4104, 520), (12, 136, 72), (16, 520, 4104), (7, 2056, 8200),
           (23, 72, 72), (24, 264, 264), (203, 72, 4104), (1030, 520, 520), (4090, 520, 72), (4090, 264, 264),
           (4090, 520, 520), (4090, 1032, 1032), (4090, 2056, 1032), (4090, 2056, 4096)]
GRADIENTS = [(23, 72, 72), (24, 264, 136), (2100, 72, 1032), (1030, 520, 520), (1030, 1032, 1032), (1030, 2056, 2056),
             (4090, 1032, 2056), (4090, 4104, 1032)]


@pytest.fixture(scope="module")
def moe():
    m = setup()
    yield m
    torch.cuda.empty_cache()


def _signs(gen, shape, each):
    return torch.randint(-1, 2, shape, generator=gen) * (torch.rand(shape, generator=gen) < each)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("dtype", base.HALVES)
@pytest.mark.parametrize("T,H,I", FORWARD)
def test_forward_of_whole_numbers_is_exact(moe, T, H, I, dtype, keep):
    """Gates of 64 and a few: from 32 on silu is the identity to the last bit (exp(-32) <
    2^-46), h = g u is exact in f32 and rounded once."""
    flush(f"dense whole numbers T={T} H={H} I={I} {dtype} keep={keep}")
    gen = torch.Generator().manual_seed(T + H + I)
    x, W = _signs(gen, (T, H), 0.75), _signs(gen, (2 * I, H), min(0.75, 27 / H))  # sums of variance 9 or less
    x[:, 0] = 1
    W[:I, 0] = 64
    Wd = _signs(gen, (H, I), 0.4)
    x, W, Wd = (gpu(v.to(dtype)) for v in (x, W, Wd))
    got = moe.moe_dense_ffn(moe.DenseWeights(W, Wd), x, keep=keep)
    y, kept = got if keep else (got, None)
    gu = x.double() @ W.double().t()
    g, u = gu[:, :I], gu[:, I:]
    assert float(g.min()) >= 32 and float(gu.abs().max()) <= 256
    if keep:
        assert torch.equal(kept, gu.to(dtype))
    h = (g * u).float().to(dtype).double()
    assert float((h.abs() @ Wd.double().abs().t()).max()) < 2 ** 24
    assert torch.equal(y, (h @ Wd.double().t()).float().to(dtype))


@pytest.mark.parametrize("dtype", base.HALVES)
@pytest.mark.parametrize("T,H,I", GRADIENTS)
def test_gradients_of_whole_numbers_are_exact(moe, T, H, I, dtype):
    flush(f"dense gradients of whole numbers T={T} H={H} I={I} {dtype}")
    base.test_gradients_of_whole_numbers_are_exact(moe, T, H, I, dtype)


def test_weight_gradients_past_32_bits(moe):
    """T 2I > 2^31: every row counts in dw_gu and dw_dn, and every row of dx."""
    T, H, I, dtype, step = 140_000, 64, 8192, torch.bfloat16, 20_000
    flush("dense gradients of whole numbers past 32 bits")
    gen = torch.Generator(device="cuda").manual_seed(3)

    def whole(lo, hi, shape):
        return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.int8).to(dtype)

    x, W, Wd = whole(-1, 1, (T, H)), whole(-1, 1, (2 * I, H)), whole(-1, 1, (H, I))
    gu = torch.empty(T, 2 * I, dtype=dtype, device="cuda")
    gu[:, :I] = 32  # silu is the identity
    gu[:, I:] = whole(-2, 2, (T, I))
    dy = torch.zeros(T, H, dtype=dtype, device="cuda")  # one or two places a row: |dh| <= 2
    at = torch.arange(T, device="cuda")
    for sign in (1, -1):
        dy[at, torch.randint(0, H, (T,), generator=gen, device="cuda")] = sign
    dx, dw_gu, dw_dn = moe.moe_dense_ffn_grad(moe.DenseWeights(W, Wd), dy, x, gu)
    want_gu = torch.zeros(2 * I, H, dtype=torch.float64, device="cuda")
    want_dn = torch.zeros(H, I, dtype=torch.float64, device="cuda")
    for a in range(0, T, step):
        rows = slice(a, a + step)
        dyr, u = dy[rows].double(), gu[rows, I:].double()
        dh = dyr @ Wd.double()
        dgu = torch.cat([dh * u, dh * 32], 1)
        ref = dgu @ W.double()
        assert float(ref.abs().max()) < 2 ** 24
        assert torch.equal(dx[rows], ref.float().to(dtype)), f"dx from row {a}"
        want_gu += dgu.t() @ x[rows].double()
        want_dn += dyr.t() @ (32 * u)
    # |terms| <= 64: no sum, finished or not, passes 64 T < 2^24
    assert torch.equal(dw_gu, want_gu.float().to(dtype)) and torch.equal(dw_dn, want_dn.float().to(dtype))
