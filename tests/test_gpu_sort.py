"""The token sort, its gradients and the routing weights' gradient on the GPU
against the fp64 oracle.

Bounds.  Copies are bitwise.  A sum of n products in f32 (fused multiply-adds,
any tree of at most n steps) is off by at most n 2^-24 of the sum of absolute
values; sigmoid(gate) by 6 2^-24 of itself (the exponential's last place, one
addition, one division, each with its propagation); then one rounding to the
rows' type."""
import numpy as np
import pytest
import torch

from _block import DTYPES, SMALL, U32, UNIT, f64, gpu, normal, permutation, rounded, within
from _gpu import flush, setup
from oracle import sort

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


# T, K, H, has_shared, gated: one token to many, one chunk to several blocks a
# row, sizes that are no multiple of a wave or a block
SIZES = [
    (1, 1, 8, False, False),
    (1, 10, 2048, True, True),
    (3, 32, 24, True, False),
    (7, 2, 4104, False, False),
    (33, 3, 520, True, True),
    (130, 13, 72, True, True),
    (257, 8, 264, False, False),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,H,has_shared,gated", SIZES)
def test_sort_and_gradients(moe, T, K, H, has_shared, gated, dtype):
    flush(f"sort T={T} K={K} H={H} shared={has_shared} gated={gated} {dtype}")
    gen = torch.Generator().manual_seed(T * 100 + K)
    S = T * K + (T if has_shared else 0)
    pos = permutation(gen, T, K, has_shared)
    skip = [s for s in (2, T * K - 1, S - 1) if T > 2]  # slots without a row
    hole = pos[skip].long()
    pos[skip] = torch.tensor([-1, T * K + 5 * T, -7], dtype=torch.int32)[:len(skip)]
    x, dout = normal(gen, (T, H), dtype), normal(gen, (T, H), dtype)
    y, dxs = normal(gen, (S, H), dtype), normal(gen, (S, H), dtype)
    w = torch.rand(T, K, generator=gen)
    gate = 3 * torch.randn(T, generator=gen) if gated else None
    fill = normal(gen, (S, H), dtype)
    n = K + 2

    xs = moe.moe_dispatch(gpu(x), gpu(pos), K, has_shared, xs=gpu(fill.clone()))
    want = sort.dispatch(f64(x), pos.numpy(), K, has_shared, f64(fill))
    assert np.array_equal(f64(xs), want)
    assert torch.equal(xs.cpu()[hole], fill[hole])  # left as they were

    dx = moe.moe_dispatch_grad(gpu(dxs), gpu(pos), K, has_shared)
    ref, mag = sort.slot_sum(f64(dxs), np.ones((T, K)), pos.numpy(), K, has_shared)
    within(dx, ref, rounded(ref, dtype, n * U32 * mag), "dx")

    out = (moe.moe_combine_gated(gpu(y), gpu(w), gpu(pos), gpu(gate), K) if gated
           else moe.moe_combine(gpu(y), gpu(w), gpu(pos), K, has_shared))
    ref, mag = sort.slot_sum(f64(y), f64(w), pos.numpy(), K, has_shared, f64(gate))
    within(out, ref, rounded(ref, dtype, (n + 6) * U32 * mag), "out")

    dy, dw, dg = moe.moe_combine_grad(gpu(dout), gpu(y), gpu(w), gpu(pos), K, has_shared, gate=gpu(gate),
                                      dy_slots=gpu(fill.clone()))
    rdy, rdw, rdg, mw, mg = sort.combine_grad(f64(dout), f64(y), f64(w), pos.numpy(), K, has_shared, f64(gate),
                                              f64(fill))
    within(dy, rdy, rounded(rdy, dtype, 8 * U32 * np.abs(rdy)), "dy")
    assert torch.equal(dy.cpu()[hole], fill[hole])
    within(dw, rdw, H * U32 * mw, "dw")
    if gated:
        # 1 - c is off by c's own error, up to 6 2^-24 absolute
        c = 1 / (1 + np.exp(-f64(gate)))
        dot = mg / np.maximum(c * (1 - c), 1e-300)
        within(dg, rdg, (H + 12) * U32 * mg + 7 * U32 * c * dot + 1e-30, "dgate")
    else:
        assert dg is None


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 512, 10), (5, 33, 32), (67, 1024, 8), (130, 64, 3)])
def test_topk_grad(moe, T, E, K):
    flush(f"topk grad T={T} E={E} K={K}")
    gen = torch.Generator().manual_seed(E)
    ids, w = moe.moe_route_topk(gpu(torch.randn(T, E, generator=gen)), K)
    dw = torch.randn(T, K, generator=gen)
    dz = moe.moe_route_topk_grad(ids, w, gpu(dw), E)
    ref, mag = sort.route_topk_grad(ids.cpu().numpy(), f64(w), f64(dw), E)
    # the mean: K products and sums; then a difference and a product
    within(dz, ref, (K + 4) * U32 * mag, "dlogits")


def test_topk_grad_with_repeated_and_foreign_ids(moe):
    ids = torch.tensor([[3, 3, 1], [7, -1, 8], [0, 2, 0]], dtype=torch.int32)
    w, dw = torch.rand(3, 3), torch.randn(3, 3)
    dz = moe.moe_route_topk_grad(gpu(ids), gpu(w), gpu(dw), 8)
    ref, mag = sort.route_topk_grad(ids.numpy(), f64(w), f64(dw), 8)
    within(dz, ref, 8 * U32 * mag, "dlogits")


def test_special_values_stay_in_their_rows(moe):
    gen = torch.Generator().manual_seed(5)
    T, K, H = 6, 2, 64
    pos = permutation(gen, T, K, True)
    y, dout = normal(gen, (T * K + T, H), torch.bfloat16), normal(gen, (T, H), torch.bfloat16)
    y[pos[2 * K].item(), 5] = float("nan")   # a slot of token 2
    dout[4, 7] = float("inf")
    w = torch.rand(T, K, generator=gen)
    out = moe.moe_combine(gpu(y), gpu(w), gpu(pos), K, True).cpu()
    assert torch.isnan(out).nonzero().tolist() == [[2, 5]]
    dy, dw, _ = moe.moe_combine_grad(gpu(dout), gpu(y), gpu(w), gpu(pos), K, True)
    bad = (~torch.isfinite(dy.cpu())).nonzero().tolist()
    rows = sorted([pos[4 * K].item(), pos[4 * K + 1].item(), pos[T * K + 4].item()])
    assert sorted(bad) == [[r, 7] for r in rows]
    assert (~torch.isfinite(dw.cpu())).nonzero().tolist() in ([[2, 0], [4, 0], [4, 1]],)


def test_combine_takes_a_longer_buffer(moe):
    gen = torch.Generator().manual_seed(6)
    T, K, H = 3, 2, 24
    pos, w = gpu(permutation(gen, T, K, False)), gpu(torch.rand(T, K, generator=gen))
    for dtype in DTYPES:
        y = gpu(normal(gen, (20, H), dtype))
        assert torch.equal(moe.moe_combine(y, w, pos, K, False), moe.moe_combine(y[:6].contiguous(), w, pos, K, False))
        with pytest.raises(ValueError, match="6 rows"):
            moe.moe_combine(y[:5], w, pos, K, False)


@pytest.mark.parametrize("gated", [False, True])
def test_combine_of_many_rows_has_the_bits_of_few(moe, gated):
    T, K, H, n = 1500, 10, 2048, 60
    flush(f"combine bits T={T} gated={gated}")
    gen = torch.Generator().manual_seed(3)
    pos = gpu(permutation(gen, T, K, True))
    pos[5::11] = -1
    y, w, gate = torch.randn(T * K + T, H, device="cuda").bfloat16(), torch.rand(T, K, device="cuda"), torch.randn(T, device="cuda")
    y[100, 3], y[200, 5] = float("nan"), float("inf")
    call = lambda y, w, pos, g: (moe.moe_combine_gated(y, w, pos, g, K) if gated  # noqa: E731
                                 else moe.moe_combine(y, w, pos, K, True))
    out = call(y, w, pos, gate)
    for t in range(0, T, n):
        slots = torch.cat([pos[t * K:(t + n) * K], pos[T * K + t:T * K + t + n]])
        few = torch.where(slots >= 0, torch.arange(len(slots), device="cuda", dtype=torch.int32), slots)
        part = call(y[slots.clamp_min(0).long()], w[t:t + n], few, gate[t:t + n])
        assert torch.equal(part.view(torch.int16), out[t:t + n].view(torch.int16))


def test_f16_overflow_and_subnormals(moe):
    T, K, H = 2, 2, 8
    pos = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    y = torch.full((4, H), 60000.0, dtype=torch.float16)
    y[2:] = 2.0 ** -20
    w = torch.tensor([[1.0, 1.0], [0.25, 0.125]])
    out = moe.moe_combine(gpu(y), gpu(w), gpu(pos), K, False).cpu()
    assert torch.isinf(out[0]).all()
    assert torch.equal(out[1].double(), torch.full((H,), 0.375 * 2.0 ** -20).double())


def test_repeated_calls_are_bitwise_equal_on_another_stream(moe):
    gen = torch.Generator().manual_seed(8)
    T, K, H = 70, 6, 1032
    pos, w = gpu(permutation(gen, T, K, True)), gpu(torch.rand(T, K, generator=gen))
    y, dout = gpu(normal(gen, (T * K + T, H), torch.float32)), gpu(normal(gen, (T, H), torch.float32))
    gate = gpu(torch.randn(T, generator=gen))
    a = moe.moe_combine_grad(dout, y, w, pos, K, True, gate=gate)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = moe.moe_combine_grad(dout, y, w, pos, K, True, gate=gate)
    s.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_python_refusals(moe):
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="multiple"):
        moe.moe_dispatch(x, pos[:7], 2, False)
    with pytest.raises(ValueError, match="shape"):
        moe.moe_dispatch(x[:3], pos, 2, False)
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_dispatch(x.t().contiguous().t(), pos, 2, False)
    with pytest.raises(ValueError, match="float32, got"):
        moe.moe_dispatch(x.double(), pos, 2, False)
    with pytest.raises(ValueError, match="int32"):
        moe.moe_dispatch(x, pos.long(), 2, False)
    with pytest.raises(ValueError, match="must be on"):
        moe.moe_dispatch(x, pos.cpu(), 2, False)
    with pytest.raises(ValueError, match="without a gate"):
        moe.moe_combine_grad(x, torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda"),
                             torch.zeros(4, 2, device="cuda"), pos, 2, False, dgate=torch.zeros(4, device="cuda"))
    with pytest.raises(moe.ops._lib.MoeError):
        moe.moe_dispatch(torch.zeros(4, 12, device="cuda"), pos, 2, False)
    assert UNIT and SMALL
