"""The dense block, the gradients' norm and clipping and the 8-bit integer products as they
run one after another, captured in a graph, on streams of their own, in every shape of the
tiles, and past 2^31 elements."""
import numpy as np
import pytest
import torch

from _block import DTYPES, SMALL, U32, UNIT, f64, gpu, normal, rounded, within
from _gpu import flush, setup
from oracle import block_norm, dense, grad_norm, int8
from test_gpu_dense import HALVES, _check_forward, _check_grad, _make
from test_gpu_int8 import _check as check_int8, _matrix

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    m = setup()
    yield m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("over", [0.1, 10.0])
@pytest.mark.parametrize("T,H,I", [(6, 72, 40), (190, 520, 264)])
def test_a_training_step_and_then_serving(moe, T, H, I, over):
    """norm, block, gradients back through both, clipping of all of them and an update; then
    the new weights in 8-bit integers.  Each stage against the oracle from its own inputs."""
    flush(f"dense chain T={T} H={H} I={I} over={over}")
    gen = torch.Generator().manual_seed(T)
    x, W, Wd = _make(gen, T, H, I, BF)
    w_pre = (torch.rand(H, generator=gen) + 0.5)
    dy, eps = normal(gen, (T, H), BF, 0.5), 1e-6
    weights = moe.DenseWeights(gpu(W), gpu(Wd))
    r, n, _, rstd = moe.moe_block_norm(gpu(x), w_pre=gpu(w_pre), eps=eps)
    y, gu = moe.moe_dense_ffn(weights, n, keep=True)
    _check_forward(y, gu, n, W, Wd, BF)
    dn, dw_gu, dw_dn = moe.moe_dense_ffn_grad(weights, gpu(dy), n, gu)
    _check_grad((dn, dw_gu, dw_dn), dy, n, gu, W, Wd, BF)
    back = moe.moe_block_norm_grad(gpu(dy), dn, r, w_pre=gpu(w_pre), rstd_pre=rstd)
    grads = [dw_gu, dw_dn] + [t for t in back if isinstance(t, torch.Tensor) and t.shape == (H,)]
    assert len(grads) == 3 and grads[2].dtype == torch.float32
    norm = moe.moe_grad_norm(grads)
    ref = grad_norm.norm([f64(g) for g in grads])
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    top = ref / over
    before = [g.clone() for g in grads]
    moe.moe_grad_clip(grads, norm, top)
    c = torch.tensor(grad_norm.factor32(float(norm), top))
    for a, b in zip(before, grads):
        assert torch.equal(b.cpu(), (a.cpu().float() * c).to(a.dtype))
    # each value keeps half a step: the norm is the limit's up to that
    after = float(moe.moe_grad_norm(grads))
    assert after <= min(ref, top) * (1 + 2.0 ** -8)
    W2, Wd2 = (v - 0.1 * g for v, g in zip((gpu(W), gpu(Wd)), grads))
    serve = moe.Int8Matrix.from_float(W2), moe.Int8Matrix.from_float(Wd2)
    for M, w in zip(serve, (W2, Wd2)):
        w = f64(w)
        assert np.all(np.abs(f64(M.codes) * f64(M.scales)[:, None] - w) <= (0.5 + 2.0 ** -15) * f64(M.scales)[:, None])
    if H % 16 or I % 16:  # 8-bit rows are whole chunks of 16
        return
    _serve(moe, n, serve)


def _serve(moe, n, serve):
    h = moe.moe_int8_linear(serve[0], n, gated=True)
    I = h.shape[1]
    z = int8.linear32(n.float().cpu().numpy(), serve[0].codes.cpu().numpy(), serve[0].scales.cpu().numpy()).astype(np.float64)
    g, u = z[:, :I], z[:, I:]
    act = dense.activate(g, u)
    within(h, act, rounded(act, BF, ((2 * np.abs(g) + 8) * 2.0 ** -23 + U32) * np.abs(act) + 2.0 ** -140), "h")
    y = moe.moe_int8_linear(serve[1], h)
    z = int8.linear32(h.float().cpu().numpy(), serve[1].codes.cpu().numpy(), serve[1].scales.cpu().numpy())
    assert torch.equal(y.cpu(), torch.from_numpy(z).to(BF))


@pytest.mark.parametrize("T", [1, 16, 300])
def test_serving_in_8_bits(moe, T):
    H, I = 528, 272
    flush(f"int8 chain T={T}")
    gen = torch.Generator().manual_seed(T)
    x, W, Wd = _make(gen, T, H, I, BF)
    _serve(moe, gpu(x), (moe.Int8Matrix.from_float(gpu(W)), moe.Int8Matrix.from_float(gpu(Wd))))


def _calls(moe, weights, M, Mg, x, dy, grads):
    y, gu = moe.moe_dense_ffn(weights, x, keep=True)
    back = moe.moe_dense_ffn_grad(weights, dy, x, gu)
    all_ = [*back[1:], *grads]
    norm = moe.moe_grad_norm(all_)
    clipped = moe.moe_grad_clip(all_, norm, 0.5, out=[torch.empty_like(g) for g in all_])
    codes, scales = moe.moe_int8_quant(x)
    z, h = moe.moe_int8_linear(M, x), moe.moe_int8_linear(Mg, x, gated=True)
    return [y, gu, *back, norm, *clipped, codes, scales, z, h]


def _setting(moe, T, H, I, seed):
    gen = torch.Generator().manual_seed(seed)
    x, W, Wd = (gpu(v) for v in _make(gen, T, H, I, BF))
    codes, scales = _matrix(gen, 2 * I, H)
    M = moe.Int8Matrix(gpu(codes), gpu(scales))
    inputs = [(gpu(normal(gen, (T, H), BF)), gpu(normal(gen, (T, H), BF)),
               [gpu(normal(gen, (n,), torch.float32)) for n in (3, 70_001)]) for _ in range(2)]
    return lambda i: _calls(moe, moe.DenseWeights(W, Wd), M, M, *inputs[i])


@pytest.mark.parametrize("T,H,I", [(1, 512, 136), (12, 2064, 136), (200, 384, 136)])
def test_graph_replays_equal_eager(moe, T, H, I):
    """All of them in one graph, replayed three times, with the program's own calls between."""
    flush(f"dense graph T={T}")
    f = _setting(moe, T, H, I, T)
    want, other = [t.clone() for t in f(0)], [t.clone() for t in f(1)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = f(0)
    for rep in range(3):
        for t in held:
            t.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        g.replay()
        again = f(1)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), f"replay {rep}"
        assert all(torch.equal(a, b) for a, b in zip(again, other)), f"eager {rep}"
    del g


@pytest.mark.parametrize("T", [4, 300])
def test_two_streams_at_once(moe, T):
    flush(f"dense streams T={T}")
    f = _setting(moe, T, 1040, 264, T)
    want = [[t.clone() for t in f(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(f(i))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


# sizes that take each tile shape and stream the operators' own tests leave out
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,H,I", [(1030, 264, 1032), (1030, 2056, 72), (1030, 520, 520), (3, 72, 4104), (12, 4104, 72),
                                   (9, 264, 8200), (1030, 136, 1032), (260, 264, 2056), (1030, 4104, 520),
                                   (4100, 520, 72), (520, 4104, 264), (260, 2056, 72), (64, 65536, 64)])
def test_other_tiles_of_the_block(moe, T, H, I, dtype):
    flush(f"dense tiles T={T} H={H} I={I} {dtype}")
    gen = torch.Generator().manual_seed(I)
    x, W, Wd = _make(gen, T, H, I, dtype)
    weights = moe.DenseWeights(gpu(W), gpu(Wd))
    y, gu = moe.moe_dense_ffn(weights, gpu(x), keep=True)
    _check_forward(y, gu, x, W, Wd, dtype)
    dy = normal(gen, (T, H), dtype, 0.5)
    _check_grad(moe.moe_dense_ffn_grad(weights, gpu(dy), gpu(x), gu), dy, x, gu, W, Wd, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,N,K", [(4100, 2064, 48), (1030, 2064, 528), (1030, 528, 1040), (1030, 2064, 272), (4100, 1040, 1040),
                                   (1030, 1040, 528), (2100, 4112, 2064), (6, 2064, 8208), (12, 2064, 16400),
                                   (2, 8208, 144), (7, 8208, 272), (5, 272, 144)])
def test_other_tiles_of_the_products_in_8_bits(moe, T, N, K, gated, dtype):
    flush(f"int8 tiles T={T} N={N} K={K} gated={gated} {dtype}")
    gen = torch.Generator().manual_seed(N)
    codes, scales = _matrix(gen, N, K)
    check_int8(moe, normal(gen, (T, K), dtype), codes, scales, gated, dtype)


def _some(T):
    """Both ends of T rows and some between."""
    return torch.tensor(sorted({0, 1, T // 3, T // 2, T - 2, T - 1}), device="cuda")


def test_block_past_32_bits(moe):
    """T 2I > 2^31 elements of the projections, and their gradients: rows of the ends and the
    middle; of the weights' gradients, sums over all rows, some lines."""
    T, H, I = 140_000, 64, 8192
    flush("dense past 32 bits")
    torch.manual_seed(1)
    x = torch.randn(T, H, device="cuda").to(BF)
    W, Wd = (torch.randn(2 * I, H, device="cuda") / 8).to(BF), (torch.randn(H, I, device="cuda") / 90).to(BF)
    dy = (torch.randn(T, H, device="cuda") / 2).to(BF)
    weights, at = moe.DenseWeights(W, Wd), _some(T)
    y, gu = moe.moe_dense_ffn(weights, x, keep=True)
    _check_forward(y[at], gu[at], x[at], W, Wd, BF)
    dx, dw_gu, dw_dn = moe.moe_dense_ffn_grad(weights, dy, x, gu)
    small = moe.moe_dense_ffn_grad(weights, dy[at], x[at], gu[at])
    _check_grad(small, dy[at], x[at], gu[at], W, Wd, BF)
    # the same sums in another order of f32, each rounded once
    err = f64(dx[at]) - f64(small[0])
    assert np.abs(err).max() <= 2 * UNIT[BF] * np.abs(f64(small[0])).max()
    # columns of the weights' gradients over all rows: dgu and h are rounded as operands, by
    # independent errors of at most U each, and T sums in f32 behind them
    cols = torch.tensor([0, 1, I // 2, I - 1], device="cuda")
    g, u = gu[:, cols].double(), gu[:, I + cols].double()
    s = torch.sigmoid(g)
    dh = dy.double() @ Wd[:, cols].double()
    for rows, d in ((cols, dh * u * s * (1 + g * (1 - s))), (I + cols, dh * g * s)):
        ref, mag = d.t() @ x.double(), d.abs().t() @ x.double().abs()
        bound = (1.5 * UNIT[BF] + 2 * 2.0 ** -14) * mag + UNIT[BF] * ref.abs() + SMALL[BF]
        assert ((dw_gu[rows].double() - ref).abs() <= bound).all()
    h = g * s * u
    ref, mag = dy.double().t() @ h, dy.double().abs().t() @ h.abs()
    assert ((dw_dn[:, cols].double() - ref).abs() <= (1.5 * UNIT[BF] + 2 * 2.0 ** -14) * mag + UNIT[BF] * ref.abs()).all()


def test_products_in_8_bits_past_32_bits(moe):
    """Rows past 2^32 elements and outputs past 2^31."""
    flush("int8 past 32 bits")
    torch.manual_seed(2)
    for T, N, K in ((70_000, 16, 65536), (270_000, 8192, 16)):
        x = torch.randn(T, K, device="cuda", dtype=BF)
        codes = torch.randint(-128, 128, (N, K), device="cuda", dtype=torch.int8)
        scales = torch.rand(N, device="cuda") + 0.5
        at, M = _some(T), moe.Int8Matrix(codes, scales)
        q, s = moe.moe_int8_quant(x)
        wq, ws = int8.quant(x[at].float().cpu().numpy())
        assert np.array_equal(q[at].cpu().numpy(), wq) and np.array_equal(s[at].cpu().numpy(), ws)
        out = moe.moe_int8_linear(M, x)
        z = int8.linear32(x[at].float().cpu().numpy(), codes.cpu().numpy(), scales.cpu().numpy())
        assert torch.equal(out[at].cpu(), torch.from_numpy(z).to(BF))
        del x, q, out


def test_a_gradient_past_32_bits(moe):
    flush("gradient past 32 bits")
    n = 2 ** 31 + 12_345
    g = torch.ones(n, device="cuda", dtype=BF)
    few = torch.full((7,), 3.0, device="cuda")
    g[-1], g[2 ** 31], g[5] = 1000.0, 2000.0, 500.0
    ref = np.sqrt(n - 3 + 1000.0 ** 2 + 2000.0 ** 2 + 500.0 ** 2 + 63)
    norm = moe.moe_grad_norm([few, g])
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    moe.moe_grad_clip([few, g], norm, 64.0)
    c = torch.tensor(grad_norm.factor32(float(norm), 64.0))
    scaled = lambda v: float((torch.tensor(v) * c).to(BF))  # noqa: E731
    assert [float(g[i]) for i in (0, 5, 2 ** 31, n - 1)] == [scaled(v) for v in (1.0, 500.0, 2000.0, 1000.0)]
    assert int((g != scaled(1.0)).sum()) == 3
    assert torch.equal(few.cpu(), torch.full((7,), 3.0) * c)


def test_clipping_refuses_tensors_that_share_memory(moe):
    g = torch.ones(64, device="cuda")
    norm, err = moe.moe_grad_norm([g, g]), moe.ops._lib.MoeError
    assert float(norm) == np.float32(np.sqrt(128.0))
    with pytest.raises(err, match="overlap"):
        moe.moe_grad_clip([g, g], norm, 1.0)
    with pytest.raises(err, match="not its own"):
        moe.moe_grad_clip([g, g], norm, 1.0, out=[g, torch.empty_like(g)])
    outs = moe.moe_grad_clip([g, g], norm, 1.0, out=[torch.empty_like(g), torch.empty_like(g)])
    assert torch.equal(outs[0], outs[1]) and torch.equal(g, torch.ones_like(g))
