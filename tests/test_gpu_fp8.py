"""Products in e4m3 with block scales on the GPU against the fp64 oracle.

Bounds.  The quantisation is bit-exact.  A product sums exact terms (8 by 8
bits) of 128 inside the matrix instruction and ceil(K/128) block sums outside,
each with two multiplications: (128 + K/128 + 4) 2^-24 of the sum of absolute
values, then one rounding.  Rows of 16 bits go through the f8 matrix
instruction, which cuts small products (oracle.fp8block.cut); rows of float32
do not.  The experts' bound adds, element by element of h,
what the neighbouring code would change where h's own error reaches a border
of e4m3 (oracle.fp8block.quant_range)."""
import numpy as np
import pytest
import torch

import oracle
from _block import DTYPES, U32, f64, gpu, normal, rounded, within
from _gpu import flush, setup
from oracle import fp8block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


def _matrix(gen, N, K):
    codes = (torch.randn(N, K, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = (torch.rand(-(-N // 128), -(-K // 128), generator=gen) + 0.5) / 100
    return codes, scales


def _w64(codes, scales):
    return fp8block.matrix(codes.double().numpy(), scales.numpy())


def _check_linear(moe, gen, T, N, K, dtype, x=None):
    codes, scales = _matrix(gen, N, K)
    x = normal(gen, (T, K), dtype) if x is None else x
    M = moe.FP8Matrix(gpu(codes), gpu(scales))
    out = moe.moe_fp8_linear(M, gpu(x))
    assert out.dtype == dtype and out.shape == (T, N)
    ref, mag = fp8block.linear(x.float().numpy(), _w64(codes, scales))
    err = (128 + -(-K // 128) + 4) * U32 * mag
    if dtype != torch.float32:
        err += _cut(x, codes, scales)
    within(out, ref, rounded(ref, dtype, err), f"linear {T} {N} {K}")
    return M, x, out


def _cut(x, codes, scales):
    return fp8block.cut(*fp8block.quant(x.float().numpy()), codes.double().numpy(), scales.numpy())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K", [(1, 16), (3, 128), (7, 144), (2, 2048), (130, 272), (5, 8208)])
def test_quant_is_bit_exact(moe, T, K, dtype):
    flush(f"quant T={T} K={K} {dtype}")
    gen = torch.Generator().manual_seed(K)
    x = normal(gen, (T, K), dtype)
    x[0, 0] = 0.0
    x[T // 2] *= 2.0 ** -7
    x[T - 1, :16] = 0
    if dtype == torch.bfloat16:
        x[0, 4], x[T - 1, 5] = 3e38, 1e-38
    q, s = moe.moe_fp8_quant(gpu(x))
    rq, rs = fp8block.quant(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.float().cpu().double().numpy(), rq)


# up to 16 rows (one launch), more (tiles), sizes around each tile's edges, K
# and N that end inside a block of 128
LINEAR = [(1, 8, 16), (1, 2048, 2048), (2, 264, 144), (8, 136, 1040), (16, 24, 4112), (15, 8200, 272), (16, 8192, 128),
          (17, 8, 16), (17, 264, 144), (33, 128, 400), (64, 520, 256), (65, 72, 2064), (200, 1032, 384),
          (300, 392, 640), (513, 136, 160), (130, 8200, 272), (700, 2056, 144), (90, 10248, 400)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,K", LINEAR)
def test_linear(moe, T, N, K, dtype):
    flush(f"linear T={T} N={N} K={K} {dtype}")
    gen = torch.Generator().manual_seed(T + N + K)
    _check_linear(moe, gen, T, N, K, dtype)


@pytest.mark.parametrize("T,N,K", [(2100, 4360, 272), (4200, 3080, 144)])
def test_linear_large(moe, T, N, K):
    """Enough tiles for the largest tile shape, all sizes ragged; the rows and
    columns compared are every 29th and 7th, and the last ones."""
    flush(f"linear large T={T} N={N} K={K}")
    gen = torch.Generator().manual_seed(T)
    codes, scales = _matrix(gen, N, K)
    x = normal(gen, (T, K), torch.bfloat16)
    out = moe.moe_fp8_linear(moe.FP8Matrix(gpu(codes), gpu(scales)), gpu(x))
    rows = sorted(set(range(0, T, 29)) | set(range(T - 40, T)))
    cols = sorted(set(range(0, N, 7)) | set(range(N - 40, N)))
    ref, mag = fp8block.linear(x.float().numpy()[rows], _w64(codes, scales)[cols])
    err = 140 * U32 * mag + fp8block.cut(*fp8block.quant(x.float().numpy()[rows]), codes.double().numpy()[cols],
                                         scales.numpy(), cols=cols)
    within(out.cpu()[rows][:, cols], ref, rounded(ref, torch.bfloat16, err), "linear large")


# a grid of each tile shape, blocks along K that do not divide among the waves,
# and the few rows that run in wide streams or in tiles
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,N,K", [(64, 2056, 1168), (130, 2056, 1040), (600, 1032, 400), (330, 4104, 1040),
                                   (500, 4104, 272), (1000, 8200, 144), (3, 4104, 2064), (5, 8200, 1040),
                                   (9, 24, 8208), (2, 6152, 4096)])
def test_linear_every_tile(moe, T, N, K, dtype):
    flush(f"linear tiles T={T} N={N} K={K} {dtype}")
    gen = torch.Generator().manual_seed(T + N)
    codes, scales = _matrix(gen, N, K)
    x = normal(gen, (T, K), dtype)
    out = moe.moe_fp8_linear(moe.FP8Matrix(gpu(codes), gpu(scales)), gpu(x))
    rows = np.unique(np.minimum(np.r_[0:T:37, 31:33, 63:65, T - 1], T - 1))
    cols = np.unique(np.minimum(np.r_[0:N:61, 31:33, 127:130, N - 9:N], N - 1))
    ref, mag = fp8block.linear(x.float().numpy()[rows], _w64(codes, scales)[cols])
    err = (128 + -(-K // 128) + 4) * U32 * mag
    if dtype != torch.float32:
        err += fp8block.cut(*fp8block.quant(x.float().numpy()[rows]), codes.double().numpy()[cols], scales.numpy(),
                            cols=cols)
    within(out.cpu()[rows][:, cols], ref, rounded(ref, dtype, err), "linear tiles")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", [(3, 24, 65536), (18, 24, 8336), (20, 24, 65536), (257, 8, 8208)])
def test_linear_long_rows(moe, T, N, K, dtype):
    """More than 64 blocks along K: several runs of weight scales, and the largest K."""
    flush(f"linear long T={T} N={N} K={K} {dtype}")
    _check_linear(moe, torch.Generator().manual_seed(T + K), T, N, K, dtype)


@pytest.mark.parametrize("T", [5, 40])
def test_gradient_by_the_input_is_the_transposed_matrix(moe, T):
    """Against the formula and against differences of the exact bilinear product."""
    gen = torch.Generator().manual_seed(2)
    N, K = 272, 400
    codes, scales = _matrix(gen, N, K)
    g = normal(gen, (T, N), torch.float32)
    Mt = moe.FP8Matrix(gpu(codes), gpu(scales)).transposed()
    dx = moe.moe_fp8_linear(Mt, gpu(g))
    W = _w64(codes, scales)
    ref, mag = fp8block.linear(g.numpy(), np.ascontiguousarray(W.T))
    within(dx, ref, (128 + 3 + 5) * U32 * mag, "dx")
    gd = fp8block.dequant_rows(*fp8block.quant(g.numpy()))
    x = np.random.default_rng(3).standard_normal((T, K))
    for t, k in ((0, 0), (T - 1, K - 1), (2, 130)):
        e = np.zeros_like(x)
        e[t, k] = 0.5
        num = (((x + e) @ W.T - (x - e) @ W.T) * gd).sum()
        assert abs(num - ref[t, k]) <= 1e-9 * mag[t, k] + 1e-12


@pytest.mark.parametrize("T", [4, 100])
def test_linear_special_rows(moe, T):
    """Zeros, tiny values, NaN and infinity: only their own rows are touched."""
    gen = torch.Generator().manual_seed(9)
    x = normal(gen, (T, 272), torch.bfloat16)
    x[0] = 0
    x[1, 128:256] = 1e-38
    x[2, 7] = float("nan")
    x[3, 200] = float("-inf")
    codes, scales = _matrix(gen, 136, 272)
    out = moe.moe_fp8_linear(moe.FP8Matrix(gpu(codes), gpu(scales)), gpu(x)).cpu()
    assert torch.equal(out[0], torch.zeros(136, dtype=torch.bfloat16))
    bad = torch.isnan(out.float())
    assert bad[2].all() and bad[3].all() and not bad[:2].any() and not bad[4:].any()
    ok = [0, 1] + list(range(4, T))
    if ok:
        ref, mag = fp8block.linear(x.float().numpy()[ok], _w64(codes, scales))
        err = 140 * U32 * mag + _cut(x[ok], codes, scales)
        within(out[ok], ref, rounded(ref, torch.bfloat16, err), "the other rows")


@pytest.mark.parametrize("T", [3, 40])
def test_nan_weights_make_their_output_columns_nan(moe, T):
    """A NaN code at the end of a row that ends inside a block of 128 stays in its column."""
    gen = torch.Generator().manual_seed(4)
    N, K = 40, 144
    codes, scales = _matrix(gen, N, K)
    codes.view(torch.uint8)[11, K - 1] = 0x7F
    codes.view(torch.uint8)[20, 0] = 0xFF
    out = moe.moe_fp8_linear(moe.FP8Matrix(gpu(codes), gpu(scales)), gpu(normal(gen, (T, K), torch.float32))).cpu()
    bad = torch.isnan(out)
    assert bad.any(0).nonzero().flatten().tolist() == [11, 20] and bad[:, [11, 20]].all()


def test_linear_repeats_bitwise_and_on_another_stream(moe):
    gen = torch.Generator().manual_seed(6)
    for T in (9, 300):
        codes, scales = _matrix(gen, 1032, 2064)
        M, x = moe.FP8Matrix(gpu(codes), gpu(scales)), gpu(normal(gen, (T, 2064), torch.float32))
        a = moe.moe_fp8_linear(M, x)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            b = moe.moe_fp8_linear(M, x)
        s.synchronize()
        assert torch.equal(a, b)


# T, E, K, H, I, shared: the two-launch path up to 16 tokens, tiles above;
# groups of one row, of several tiles, empty ones
EXPERTS = [(1, 8, 2, 256, 128, False), (4, 8, 2, 256, 128, True), (8, 64, 10, 384, 256, True), (16, 3, 3, 128, 384, True),
           (17, 8, 2, 256, 128, False), (40, 64, 10, 384, 256, True), (200, 4, 2, 128, 128, True),
           (300, 5, 1, 640, 384, False), (3, 64, 10, 256, 128, True), (8, 64, 8, 128, 640, False)]


def _bank(gen, E, H, I, shared):
    G = E + int(shared)
    gu, dn = _matrix(gen, G * 2 * I, H), _matrix(gen, G * H, I)
    return (gu[0].view(G, 2 * I, H), gu[1].view(G, 2 * I // 128, H // 128) * (H / 100) ** -0.5,
            dn[0].view(G, H, I), dn[1].view(G, H // 128, I // 128) * (I / 100) ** -0.5)


def _check_experts(moe, bank, x, ids, E, H, I, shared, **kw):
    T, K = ids.shape
    counts, offsets, sorted_slot, slot_pos, groups = moe.moe_permute(gpu(ids), E, shared)
    W = moe.FP8Weights(*(gpu(b) for b in bank), E, H, I, shared)
    y = moe.moe_fp8_expert_ffn(W, gpu(x), K, offsets, sorted_slot, groups, **kw)
    off, slots = offsets.cpu().numpy(), sorted_slot.cpu().numpy()
    got = f64(y)
    for g in range(E + int(shared)):
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        rows = slots[a:b] // K if g < E else slots[a:b] - T * K
        ref, err = fp8block.expert(x.float().numpy()[rows], (bank[0][g].double().numpy(), bank[1][g].numpy()),
                                   (bank[2][g].double().numpy(), bank[3][g].numpy()), I)
        within(got[a:b], ref, rounded(ref, torch.bfloat16, err), f"group {g}")
    return y, (offsets, sorted_slot, slot_pos, groups)


@pytest.mark.parametrize("T,E,K,H,I,shared", EXPERTS)
def test_experts(moe, T, E, K, H, I, shared):
    flush(f"fp8 experts T={T} E={E} K={K} H={H} I={I} shared={shared}")
    gen = torch.Generator().manual_seed(T + E)
    bank = _bank(gen, E, H, I, shared)
    x = normal(gen, (T, H), torch.bfloat16)
    z = torch.randn(T, E, generator=gen) + torch.randn(E, generator=gen)
    ids = torch.topk(z, K, dim=1).indices.int()
    _check_experts(moe, bank, x, ids, E, H, I, shared)


# enough row tiles that a block takes two column tiles in a row, of gate_up with
# a single block along K, and of down with one and with two
@pytest.mark.parametrize("T,E,K,H,I", [(100, 512, 8, 128, 1024), (60, 320, 10, 2048, 128), (80, 512, 8, 1024, 256)])
def test_experts_many_groups(moe, T, E, K, H, I):
    flush(f"fp8 experts, many groups T={T} E={E} H={H} I={I}")
    torch.manual_seed(T)
    codes = lambda *s: (torch.randn(s, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    bank = (codes(E + 1, 2 * I, H), (torch.rand(E + 1, 2 * I // 128, H // 128, device="cuda") + 0.5) / (100 * H ** 0.5),
            codes(E + 1, H, I), (torch.rand(E + 1, H // 128, I // 128, device="cuda") + 0.5) / (100 * I ** 0.5))
    x = torch.randn(T, H, device="cuda").bfloat16()
    ids = torch.topk(torch.randn(T, E, device="cuda"), K, dim=1).indices.int()
    ids[:, 0] = 3  # one group of several rows tiles' worth
    counts, offsets, ss, pos, groups = moe.moe_permute(ids, E, True)
    y = f64(moe.moe_fp8_expert_ffn(moe.FP8Weights(*bank, E, H, I, True), x, K, offsets, ss, groups))
    off, slots = offsets.cpu().numpy(), ss.cpu().numpy()
    xf = x.float().cpu().numpy()
    for g in [0, 1, 3, E // 2, E - 1, E]:
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        rows = slots[a:b] // K if g < E else slots[a:b] - T * K
        w = [(c[g].double().cpu().numpy(), s[g].cpu().numpy()) for c, s in (bank[:2], bank[2:])]
        ref, err = fp8block.expert(xf[rows], w[0], w[1], I)
        within(y[a:b], ref, rounded(ref, torch.bfloat16, err), f"group {g}")
    assert np.isfinite(y).all()


@pytest.mark.parametrize("T", [12, 60])
def test_experts_with_repeated_and_foreign_ids(moe, T):
    """An expert named twice for a token gets two rows (more than 16 in a decode
    batch's group); an id outside the bank belongs to no group."""
    E, K, H, I = 4, 3, 256, 128
    gen = torch.Generator().manual_seed(T)
    bank = _bank(gen, E, H, I, True)
    x = normal(gen, (T, H), torch.bfloat16)
    ids = torch.full((T, K), 2, dtype=torch.int32)
    ids[0], ids[1, 1], ids[T - 1, 2] = -1, 7, 0
    y0 = torch.full((T * K + T, H), 5.0, dtype=torch.bfloat16, device="cuda")
    # the shared group starts behind the routed rows that exist
    y, (offsets, *_ ) = _check_experts(moe, bank, x, ids, E, H, I, True, y_slots=y0)
    end = int(offsets[-1])
    assert torch.equal(y[end:], torch.full_like(y[end:], 5.0))


def test_expert_rows_with_nan_stay_alone(moe):
    for T in (6, 60):
        E, K, H, I = 8, 2, 256, 128
        gen = torch.Generator().manual_seed(T)
        bank = _bank(gen, E, H, I, True)
        x = normal(gen, (T, H), torch.bfloat16)
        x[3, 200] = float("nan")
        ids = torch.topk(torch.randn(T, E, generator=gen), K, dim=1).indices.int()
        _, offsets, sorted_slot, slot_pos, groups = moe.moe_permute(gpu(ids), E, True)
        W = moe.FP8Weights(*(gpu(b) for b in bank), E, H, I, True)
        y = moe.moe_fp8_expert_ffn(W, gpu(x), K, offsets, sorted_slot, groups).cpu()
        mine = sorted(slot_pos.cpu()[[3 * K, 3 * K + 1, T * K + 3]].tolist())
        assert torch.isnan(y.float()).any(1).nonzero().flatten().tolist() == mine
        assert torch.isnan(y.float())[mine].all()


def test_python_refusals(moe):
    M = moe.FP8Matrix(torch.zeros(16, 32, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda"))
    x = torch.zeros(4, 32, device="cuda")
    with pytest.raises(ValueError, match=r"\[T, 32\]"):
        moe.moe_fp8_linear(M, x[:, :16].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_fp8_linear(M, torch.zeros(32, 4, device="cuda").t())
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_fp8_linear(M, torch.zeros(20, 32, device="cuda"), ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="scales"):
        moe.moe_fp8_linear(moe.FP8Matrix(M.codes, torch.ones(1, 2, device="cuda")), x)
    with pytest.raises(ValueError, match="uint8"):
        moe.moe_fp8_linear(moe.FP8Matrix(M.codes.int(), M.scales), x)
    with pytest.raises(moe.ops._lib.MoeError, match="multiple of 16"):
        moe.moe_fp8_quant(torch.zeros(2, 24, device="cuda"))
    assert oracle
