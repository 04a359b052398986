"""The operators in a row, as a block uses them, and under HIP graph capture.

Training: route -> permute -> dispatch -> the caller's own experts -> gated
combine -> norm, gate and residual -> the next norm, and every gradient back to
the inputs, against torch's autograd of the same formulas in float64 on the CPU.
All rows are float32.  A value passes through fewer than 2^13 roundings of at
most 2^-24 on its way (the longest sums: 96 columns, 40 tokens, twice each way),
none after a cancellation that the outputs' norm does not share: 2^-11 of the
norm.

Serving: norm -> router -> permute -> e4m3 experts -> gated combine -> norm and
residual, each stage against its oracle on the stage before's own output.
"""
import numpy as np
import pytest
import torch

import oracle
from _block import U32, f64, normal, rounded, within
from _gpu import flush, setup
from oracle import block_norm, fp8block, sort
from workloads import make_router

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


def _rel(a, b):
    return float(np.linalg.norm(f64(a) - b) / max(np.linalg.norm(b), 1e-30))


def test_training_step_of_a_block(moe):
    gen = torch.Generator().manual_seed(0)
    T, E, K, H = 40, 6, 3, 96
    a, b, eps = 0.9, 0.7, 1e-5
    x = normal(gen, (T, H), torch.float32)
    res, wr = normal(gen, (T, H), torch.float32), normal(gen, (H, E), torch.float32, H ** -0.5)
    We, Ws = normal(gen, (E, H, H), torch.float32, H ** -0.5), normal(gen, (H, H), torch.float32, H ** -0.5)
    gate, w_post, w_pre = torch.randn(T, generator=gen), torch.rand(H, generator=gen) + 0.5, torch.rand(H, generator=gen) + 0.5
    cr, cn = normal(gen, (T, H), torch.float32), normal(gen, (T, H), torch.float32)
    logits = x @ wr

    # forward on the GPU
    d = lambda t: t.cuda()  # noqa: E731
    ids, w = moe.moe_route_topk(d(logits), K)
    counts, offsets, _, pos, _ = moe.moe_permute(ids, E, True)
    off = offsets.cpu().tolist()
    xs = moe.moe_dispatch(d(x), pos, K, True)
    mats = [d(We[e]) for e in range(E)] + [d(Ws)]
    y = torch.cat([xs[off[g]:off[g + 1]] @ mats[g] for g in range(E + 1)])
    out = moe.moe_combine_gated(y, w, pos, d(gate), K)
    r, n, sp, sn = moe.moe_block_norm(d(res), out, w_post=d(w_post), w_pre=d(w_pre), res_scale=a, out_scale=b, eps=eps)

    # and back
    dres, dout, _, dw_post, dw_pre = moe.moe_block_norm_grad(
        d(cr), d(cn), r, out, w_post=d(w_post), w_pre=d(w_pre), rstd_post=sp, rstd_pre=sn, res_scale=a, out_scale=b)
    dy, dw, dgate = moe.moe_combine_grad(dout, y, w, pos, K, True, gate=d(gate))
    dlogits = moe.moe_route_topk_grad(ids, w, dw, E)
    dxs = torch.cat([dy[off[g]:off[g + 1]] @ mats[g].t().contiguous() for g in range(E + 1)])
    dx = moe.moe_dispatch_grad(dxs, pos, K, True)

    # the same in float64 with torch's autograd
    v = {k: t.double().requires_grad_() for k, t in
         dict(x=x, z=logits, res=res, gate=gate, w_post=w_post, w_pre=w_pre).items()}
    idc = ids.cpu().long()
    p = torch.softmax(torch.gather(v["z"], 1, idc), 1)
    each = torch.einsum("th,ehj->tej", v["x"], We.double())
    o = (torch.gather(each, 1, idc[..., None].expand(-1, -1, H)) * p[..., None]).sum(1)
    o = o + torch.sigmoid(v["gate"])[:, None] * (v["x"] @ Ws.double())
    u = o * (o.square().mean(1, keepdim=True) + eps).rsqrt() * v["w_post"]
    r64 = a * v["res"] + b * u
    n64 = r64 * (r64.square().mean(1, keepdim=True) + eps).rsqrt() * v["w_pre"]
    ((r64 * cr.double()).sum() + (n64 * cn.double()).sum()).backward()
    got = dict(x=dx, z=dlogits, res=dres, gate=dgate, w_post=dw_post, w_pre=dw_pre)
    for name, g in got.items():
        assert _rel(g, v[name].grad.numpy()) <= 2.0 ** -11, name
    assert _rel(n, n64.detach().numpy()) <= 2.0 ** -11


@pytest.mark.parametrize("T", [3, 50])
def test_serving_step_of_a_block(moe, T):
    flush(f"serving step T={T}")
    gen = torch.Generator().manual_seed(T)
    E, K, H, I = 16, 4, 256, 128
    rb = make_router(E, H, True, seed=1)
    R = moe.NVFP4Router.from_bank(rb)
    codes = lambda *s: (torch.randn(s, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    gu, gus = codes(E + 1, 2 * I, H), torch.rand(E + 1, 2 * I // 128, H // 128, generator=gen) / 1000 + 5e-4
    dn, dns = codes(E + 1, H, I), torch.rand(E + 1, H // 128, I // 128, generator=gen) / 1000 + 5e-4
    W = moe.FP8Weights(gu.cuda(), gus.cuda(), dn.cuda(), dns.cuda(), E, H, I, True)
    res = normal(gen, (T, H), torch.bfloat16, 2.0)
    w1, w2, w3 = (torch.rand(H, generator=gen) + 0.5 for _ in range(3))

    x0 = res.cuda()
    _, x, _, _ = moe.moe_block_norm(x0, w_pre=w1.cuda())
    ids, w, z, gate = moe.moe_router_topk(R, x, K)
    counts, offsets, ss, pos, groups = moe.moe_permute(ids, E, True)
    y = moe.moe_fp8_expert_ffn(W, x, K, offsets, ss, groups)
    out = moe.moe_combine_gated(y, w, pos, gate, K)
    r, n, _, _ = moe.moe_block_norm(x0, out, w_post=w2.cuda(), w_pre=w3.cuda())

    eps = float(np.float32(1e-6))
    ref, _ = block_norm.pre(f64(res), f64(w1), eps)
    within(x, ref, rounded(ref, torch.bfloat16, 40 * U32 * np.abs(ref)), "x")
    assert np.array_equal(ids.cpu().numpy(), oracle.route_topk(z.cpu().numpy(), K)[0])
    off, slots = offsets.cpu().numpy(), ss.cpu().numpy()
    for g in range(E + 1):
        lo, hi = off[g], off[g + 1]
        if lo == hi:
            continue
        rows = slots[lo:hi] // K if g < E else slots[lo:hi] - T * K
        ref, err = fp8block.expert(x.float().cpu().numpy()[rows], (gu[g].double().numpy(), gus[g].numpy()),
                                   (dn[g].double().numpy(), dns[g].numpy()), I)
        within(y[lo:hi], ref, rounded(ref, torch.bfloat16, err), f"group {g}")
    ref, mag = sort.slot_sum(f64(y), f64(w), pos.cpu().numpy(), K, True, f64(gate))
    within(out, ref, rounded(ref, torch.bfloat16, (K + 8) * U32 * mag), "out")
    ref, _, u = block_norm.post(f64(res), f64(out), None, f64(w2), 1.0, 1.0, eps)
    within(r, ref, rounded(ref, torch.bfloat16, 48 * U32 * u + 3 * U32 * np.abs(f64(res))), "r")
    ref, _ = block_norm.pre(f64(r), f64(w3), eps)
    within(n, ref, rounded(ref, torch.bfloat16, 40 * U32 * np.abs(ref)), "n")


def _tensors(v):
    if isinstance(v, torch.Tensor):
        return [v]
    return [t for x in (v or ()) for t in _tensors(x)]


@pytest.mark.parametrize("T", [5, 200])
def test_graph_replays_equal_eager(moe, T):
    """Every operator captured in one graph and replayed three times, with the
    program's own eager calls of them between the replays."""
    flush(f"graph T={T}")
    gen = torch.Generator().manual_seed(T)
    E, K, H, I = 16, 4, 384, 128
    S = T * K + T
    c = lambda *s, dt=torch.bfloat16: normal(gen, s, dt).cuda()  # noqa: E731
    x, y, dxs, dout, res = c(T, H), c(S, H), c(S, H), c(T, H), c(T, H)
    gate, w1, w2 = c(T, dt=torch.float32), c(H, dt=torch.float32), c(H, dt=torch.float32)
    ids, w = moe.moe_route_topk(c(T, E, dt=torch.float32), K)
    _, offsets, ss, pos, groups = moe.moe_permute(ids, E, True)
    codes = lambda *s: (torch.randn(s, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda()  # noqa: E731
    M = moe.FP8Matrix(codes(264, H), torch.rand(3, 3, generator=gen).cuda())
    W = moe.FP8Weights(codes(E + 1, 2 * I, H), torch.rand(E + 1, 2, 3, generator=gen).cuda() / 500,
                       codes(E + 1, H, I), torch.rand(E + 1, 3, 1, generator=gen).cuda() / 500, E, H, I, True)

    def calls(x, res):
        xs = moe.moe_dispatch(x, pos, K, True)
        dx = moe.moe_dispatch_grad(dxs, pos, K, True)
        cg = moe.moe_combine_grad(dout, y, w, pos, K, True, gate=gate)
        dz = moe.moe_route_topk_grad(ids, w, cg[1], E)
        bn = moe.moe_block_norm(res, x, gate=gate, w_post=w1, w_pre=w2)
        bg = moe.moe_block_norm_grad(dout, x, bn[0], x, gate=gate, w_post=w1, w_pre=w2, rstd_post=bn[2], rstd_pre=bn[3])
        q = moe.moe_fp8_quant(x)
        z = moe.moe_fp8_linear(M, x)
        e = moe.moe_fp8_expert_ffn(W, x, K, offsets, ss, groups)
        return _tensors([xs, dx, cg, dz, bn, bg, [t.view(torch.uint8) for t in q], z, e])

    bits = lambda t: t.view(torch.uint8) if t.dtype != torch.uint8 else t  # noqa: E731
    want = [t.clone() for t in calls(x, res)]
    x2, res2 = c(T, H), c(T, H)
    other = [t.clone() for t in calls(x2, res2)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = calls(x, res)
    for rep in range(3):
        for t in held:
            bits(t).fill_(0x5A)
        torch.cuda.synchronize()
        g.replay()
        again = calls(x2, res2)
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(held, want)):
            assert torch.equal(bits(p), bits(q)), f"replay {rep}, output {i}"
        for i, (p, q) in enumerate(zip(again, other)):
            assert torch.equal(bits(p), bits(q)), f"eager {rep}, output {i}"
    del g


def test_two_streams_at_once(moe):
    """The same operators on two streams without ordering between them."""
    gen = torch.Generator().manual_seed(2)
    T, H, N = 300, 2064, 520
    x = [normal(gen, (T, H), torch.bfloat16).cuda() for _ in range(2)]
    M = moe.FP8Matrix((torch.randn(N, H, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).cuda(),
                      torch.rand(-(-N // 128), -(-H // 128), generator=gen).cuda())
    w = torch.rand(H, generator=gen).cuda()
    f = lambda t: (moe.moe_fp8_linear(M, t), *moe.moe_block_norm(t, w_pre=w)[1:2])  # noqa: E731
    want = [[o.clone() for o in f(t)] for t in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(f(x[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for p, q in zip(outs, want[i]):
                assert torch.equal(p, q)
