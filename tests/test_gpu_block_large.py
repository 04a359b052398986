"""Rows past 2^31 elements and 4 GiB: the sort, norm and e4m3 operators at sizes
whose offsets pass 32 bits, on sampled rows (the first, the last, the ones
around the borders) against the fp64 oracles.  Bounds as in the operators' own
tests."""
import numpy as np
import pytest
import torch

from _block import U32, f64, rounded, within
from _gpu import flush, setup
from oracle import block_norm, fp8block, sort

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    m = setup()
    yield m
    torch.cuda.empty_cache()


def _normal(*shape, dtype=BF):
    return torch.randn(shape, device="cuda", dtype=dtype)


def _around(n, width):
    """Rows of [n, width]: both ends, and those at 2^31 and 2^32 elements and bytes of bf16."""
    rows = {0, 1, n - 1, n - 2}
    for border in (2 ** 30, 2 ** 31, 2 ** 32):
        rows |= {border // width + d for d in (-1, 0, 1)}
    return torch.tensor(sorted(r for r in rows if 0 <= r < n), device="cuda")


def test_sort_past_32_bits(moe):
    T, K, H = 50_000, 10, 4096
    flush(f"large sort T={T} K={K} H={H}")
    torch.manual_seed(0)
    S = T * K + T
    pos = torch.cat([torch.randperm(T * K, device="cuda"), T * K + torch.randperm(T, device="cuda")]).int()
    slot_of = torch.empty(S, dtype=torch.long, device="cuda")
    slot_of[pos.long()] = torch.arange(S, device="cuda")
    x, w, gate = _normal(T, H), torch.rand(T, K, device="cuda"), _normal(T, dtype=torch.float32)
    xs = moe.moe_dispatch(x, pos, K, True)
    at = _around(S, H)
    tok = torch.where(slot_of[at] < T * K, slot_of[at] // K, slot_of[at] - T * K)
    assert torch.equal(xs[at], x[tok])
    tokens = torch.cat([tok, torch.tensor([0, T - 1], device="cuda")])
    small = torch.cat([torch.arange(len(tokens) * K, device="cuda"),
                       len(tokens) * K + torch.arange(len(tokens), device="cuda")]).int().cpu().numpy()
    slots = torch.cat([(tokens[:, None] * K + torch.arange(K, device="cuda")).reshape(-1), T * K + tokens])
    rows = f64(xs[pos.long()[slots]])  # the tokens' slot rows, in slot order
    ones = np.ones((len(tokens), K))
    dx = moe.moe_dispatch_grad(xs, pos, K, True)
    ref, mag = sort.slot_sum(rows, ones, small, K, True)
    within(dx[tokens], ref, rounded(ref, BF, (K + 2) * U32 * mag), "dx")
    out = moe.moe_combine_gated(xs, w, pos, gate, K)
    ref, mag = sort.slot_sum(rows, f64(w[tokens]), small, K, True, f64(gate[tokens]))
    within(out[tokens], ref, rounded(ref, BF, (K + 8) * U32 * mag), "out")
    dout = _normal(T, H)
    dy, dw, dg = moe.moe_combine_grad(dout, xs, w, pos, K, True, gate=gate)
    rdy, rdw, _, mw, _ = sort.combine_grad(f64(dout[tokens]), rows, f64(w[tokens]), small, K, True, f64(gate[tokens]),
                                           np.zeros_like(rows))
    within(dy[pos.long()[slots]], rdy, rounded(rdy, BF, 8 * U32 * np.abs(rdy)), "dy")
    within(dw[tokens], rdw, H * U32 * mw, "dw")
    assert torch.isfinite(dg).all()


def test_topk_grad_past_32_bits(moe):
    T, E, K = 4_200_000, 512, 2
    flush(f"large topk_grad T={T} E={E}")
    torch.manual_seed(1)
    ids = torch.stack([torch.randint(0, 256, (T,), device="cuda"), torch.randint(256, 512, (T,), device="cuda")], 1).int()
    w = torch.softmax(_normal(T, K, dtype=torch.float32), 1)
    dw = _normal(T, K, dtype=torch.float32)
    dz = moe.moe_route_topk_grad(ids, w, dw, E)
    at = _around(T, E)
    ref, mag = sort.route_topk_grad(ids[at].cpu().numpy(), f64(w[at]), f64(dw[at]), E)
    within(dz[at], ref, (K + 4) * U32 * mag, "dlogits")
    assert int((dz != 0).sum(dtype=torch.int64)) <= T * K


def test_norm_past_32_bits(moe):
    T, H, a, b = 270_000, 8192, 0.9, 0.6
    flush(f"large norm T={T} H={H}")
    torch.manual_seed(2)
    res, y, gate = _normal(T, H), _normal(T, H), _normal(T, dtype=torch.float32)
    w_post, w_pre = _normal(H, dtype=torch.float32), _normal(H, dtype=torch.float32)
    r, n, sp, sn = moe.moe_block_norm(res, y, gate=gate, w_post=w_post, w_pre=w_pre, res_scale=a, out_scale=b)
    at = _around(T, H)
    a, b, eps = float(np.float32(a)), float(np.float32(b)), float(np.float32(1e-6))
    g64, wq, wn = f64(gate[at]), f64(w_post), f64(w_pre)
    ref, rsp, u = block_norm.post(f64(res[at]), f64(y[at]), g64, wq, a, b, eps)
    within(r[at], ref, rounded(ref, BF, 48 * U32 * u + 3 * U32 * np.abs(a * f64(res[at]))), "r")
    within(sp[at], rsp, 32 * U32 * rsp, "rstd_post")
    ref, rsn = block_norm.pre(f64(r[at]), wn, eps)
    within(n[at], ref, rounded(ref, BF, 40 * U32 * np.abs(ref)), "n")
    dr, dn = res, n  # any rows serve
    dres, dy, dg, dw_post, dw_pre = moe.moe_block_norm_grad(dr, dn, r, y, gate=gate, w_post=w_post, w_pre=w_pre,
                                                            rstd_post=sp, rstd_pre=sn, res_scale=a, out_scale=b)
    args = (f64(dr[at]), f64(dn[at]), f64(r[at]), f64(y[at]), g64, wq, wn, f64(sp[at]), f64(sn[at]), a, b)
    ref, mag = block_norm.grad(*args), block_norm.grad(*args, magnitudes=True)
    for name, t in (("dres", dres), ("dy", dy)):
        within(t[at], ref[name], rounded(ref[name], BF, 72 * U32 * mag[name]), name)
    # the sum over the tokens, of some columns: a block adds up to 270000 / 1024
    # rows, then 1024 / 32 partial rows to a share and 32 shares
    cols = torch.tensor([0, 5, 4097, 8191], device="cuda")
    terms = dn[:, cols].double() * r[:, cols].double() * sn.double()[:, None]
    within(dw_pre[cols], f64(terms.sum(0)), (264 + 64 + 4) * U32 * f64(terms.abs().sum(0)), "dw_pre")
    assert torch.isfinite(dw_post).all() and torch.isfinite(dg).all()


def _codes(*shape):
    return (torch.randn(shape, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)


def test_linear_past_32_bits(moe):
    T, N, K = 66_000, 32_800, 144
    flush(f"large linear T={T} N={N} K={K}")
    torch.manual_seed(3)
    codes, scales = _codes(N, K), (torch.rand(-(-N // 128), 2, device="cuda") + 0.5) / 100
    x = _normal(T, K)
    out = moe.moe_fp8_linear(moe.FP8Matrix(codes, scales), x)
    at = _around(T, N)
    cols = np.r_[0:40, 16300:16340, N - 40:N]
    c, s = codes.float().cpu(), scales.cpu()
    W = fp8block.matrix(c.double().numpy(), s.numpy())[cols]
    xr = x[at].float().cpu().numpy()
    ref, mag = fp8block.linear(xr, W)
    err = (128 + 2 + 4) * U32 * mag + fp8block.cut(*fp8block.quant(xr), c.double().numpy()[cols], s.numpy(), cols=cols)
    within(out[at][:, torch.from_numpy(cols).cuda()], ref, rounded(ref, BF, err), "out")


def test_experts_past_32_bits(moe):
    T, E, K, H, I = 30_000, 12, 10, 8192, 128
    flush(f"large experts T={T} E={E} K={K} H={H} I={I}")
    torch.manual_seed(4)
    bank = (_codes(E + 1, 2 * I, H), (torch.rand(E + 1, 2 * I // 128, H // 128, device="cuda") + 0.5) / (100 * H ** 0.5),
            _codes(E + 1, H, I), (torch.rand(E + 1, H // 128, I // 128, device="cuda") + 0.5) / (100 * I ** 0.5))
    x = _normal(T, H)
    ids = torch.topk(_normal(T, E, dtype=torch.float32), K, dim=1).indices.int()
    _, offsets, ss, pos, groups = moe.moe_permute(ids, E, True)
    y = moe.moe_fp8_expert_ffn(moe.FP8Weights(*bank, E, H, I, True), x, K, offsets, ss, groups)
    off = offsets.cpu().numpy()
    at = _around(T * K + T, H)
    for p in at.cpu().tolist():
        g = int(np.searchsorted(off, p, side="right")) - 1
        slot = int(ss[p])
        row = slot // K if g < E else slot - T * K
        w = [(c[g].double().cpu().numpy(), s[g].cpu().numpy()) for c, s in (bank[:2], bank[2:])]
        ref, err = fp8block.expert(x[row:row + 1].float().cpu().numpy(), w[0], w[1], I)
        within(y[p:p + 1], ref, rounded(ref, BF, err), f"row {p}")
