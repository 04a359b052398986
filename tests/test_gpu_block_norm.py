"""The norms before and after a block on the GPU against the fp64 oracle.

Bounds.  A row's sums run over at most 32 values per lane, then 6 steps over
the wave and 8 over the waves: 46 roundings of positive terms in rstd, whose
root halves them, so rstd is good to 32 2^-24 with its own division and root;
a product with it to 40 2^-24.  sigmoid: 6 2^-24.  The gradients' formulas have
fewer than 64 roundings on any path from an input to an output of a row, each
on a partial result no larger than the same formula of absolute values; the
sums over tokens add the rows of a block and the joins."""
import numpy as np
import pytest
import torch

from _block import DTYPES, U32, f64, gpu, normal, rounded, within
from _gpu import flush, setup
from oracle import block_norm as ora

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    return setup()


def _inputs(T, H, dtype, gate, post, pre, seed=0):
    gen = torch.Generator().manual_seed(seed + T)
    v = dict(res=normal(gen, (T, H), dtype, 3.0), y=normal(gen, (T, H), dtype))
    v["gate"] = (None if gate == "none" else torch.randn(T, generator=gen) * 2 if gate == "token"
                 else normal(gen, (T, H), dtype, 2.0))
    v["w_post"] = torch.randn(H, generator=gen) if post else None
    v["w_pre"] = torch.randn(H, generator=gen) if pre else None
    v["dr"], v["dn"] = normal(gen, (T, H), dtype), normal(gen, (T, H), dtype) if pre else None
    return v


def _check(moe, v, dtype, a, b, eps=EPS):
    d = {k: gpu(t) for k, t in v.items()}
    n64 = {k: f64(t) for k, t in v.items()}
    r, n, sp, sn = moe.moe_block_norm(d["res"], d["y"], gate=d["gate"], w_post=d["w_post"], w_pre=d["w_pre"],
                                      res_scale=a, out_scale=b, eps=eps)
    a, b = float(np.float32(a)), float(np.float32(b))
    eps = float(np.float32(eps))
    ref, rsp, u = ora.post(n64["res"], n64["y"], n64["gate"], n64["w_post"], a, b, eps)
    within(r, ref, rounded(ref, dtype, 48 * U32 * u + 3 * U32 * np.abs(a * n64["res"])), "r")
    if v["w_post"] is not None:
        within(sp, rsp, 32 * U32 * rsp, "rstd_post")
    else:
        assert sp is None
    r64 = f64(r)  # the second norm is that of the stored rows
    if v["w_pre"] is not None:
        ref, rsn = ora.pre(r64, n64["w_pre"], eps)
        within(sn, rsn, 32 * U32 * rsn, "rstd_pre")
        within(n, ref, rounded(ref, dtype, 40 * U32 * np.abs(ref)), "n")
    else:
        assert n is None and sn is None
    got = moe.moe_block_norm_grad(d["dr"], d["dn"], r, d["y"], gate=d["gate"], w_post=d["w_post"],
                                  w_pre=d["w_pre"], rstd_post=sp, rstd_pre=sn, res_scale=a, out_scale=b)
    args = (n64["dr"], n64["dn"], r64, n64["y"], n64["gate"], n64["w_post"], n64["w_pre"], f64(sp), f64(sn), a, b)
    ref, mag = ora.grad(*args), ora.grad(*args, magnitudes=True)
    T = v["res"].shape[0]
    over_tokens = 64 + 64  # a block's rows, the blocks of a share, the shares
    for name, t in zip(("dres", "dy", "dgate", "dw_post", "dw_pre"), got):
        if name not in ref:
            assert t is None, name
            continue
        if name.startswith("dw"):
            within(t, ref[name], over_tokens * U32 * mag[name] + 1e-37, name)
        elif name == "dgate" and v["gate"].dim() == 1:
            # 1 - c is off by up to 7 2^-24 absolute
            c = 1 / (1 + np.exp(-n64["gate"]))
            within(t, ref[name], (72 + 7 / np.maximum(1 - c, 1e-30)) * U32 * mag[name] + 1e-37, name)
        elif name == "dgate":
            c = 1 / (1 + np.exp(-n64["gate"]))
            within(t, ref[name], rounded(ref[name], dtype, (72 + 7 / np.maximum(1 - c, 1e-30)) * U32 * mag[name]), name)
        else:
            within(t, ref[name], rounded(ref[name], dtype, 72 * U32 * mag[name]), name)
    return r, n, got


# one row to many; one chunk of a lane to eight waves a row, each shape's edge
# and one past it
SIZES = [(1, 8), (5, 2048), (3, 520), (9, 264), (700, 512), (515, 1032), (2, 2056), (6, 4104), (3, 8192), (4, 8184),
         (2100, 24), (513, 2048)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_all_parts(moe, T, H, dtype):
    flush(f"block norm T={T} H={H} {dtype}")
    _check(moe, _inputs(T, H, dtype, "token", True, True), dtype, 0.9, 0.6)


@pytest.mark.parametrize("gate", ["none", "token", "element"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T,H", [(6, 264), (9, 2048), (600, 136), (5, 4128)])
def test_parts(moe, T, H, post, pre, gate):
    flush(f"block norm T={T} H={H} post={post} pre={pre} gate={gate}")
    for dtype in (torch.bfloat16, torch.float32):
        _check(moe, _inputs(T, H, dtype, gate, post, pre, seed=3), dtype, -1.25, 0.5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H", [(1, 16), (5, 2048), (700, 264), (3, 8192)])
def test_norm_alone(moe, T, H, dtype):
    """Without y: the norm before a first block, and its gradient with and without dr."""
    gen = torch.Generator().manual_seed(1)
    res, w, dn = normal(gen, (T, H), dtype), torch.randn(H, generator=gen), normal(gen, (T, H), dtype)
    dr = normal(gen, (T, H), dtype)
    x = gpu(res)
    r, n, sp, sn = moe.moe_block_norm(x, w_pre=gpu(w))
    assert r is x and sp is None
    ref, rs = ora.pre(f64(res), f64(w), float(np.float32(1e-6)))
    within(n, ref, rounded(ref, dtype, 40 * U32 * np.abs(ref)), "n")
    for g in (dr, None):
        got = moe.moe_block_norm_grad(gpu(g), gpu(dn), x, w_pre=gpu(w), rstd_pre=sn)
        assert got[1] is None and got[2] is None and got[3] is None
        args = (f64(g), f64(dn), f64(res), None, None, None, f64(w), None, f64(sn), 1.0, 1.0)
        ref, mag = ora.grad(*args), ora.grad(*args, magnitudes=True)
        within(got[0], ref["dres"], rounded(ref["dres"], dtype, 72 * U32 * mag["dres"]), "dres")
        within(got[4], ref["dw_pre"], 130 * U32 * mag["dw_pre"] + 1e-37, "dw_pre")


def test_rows_of_zeros_and_of_extremes(moe):
    for dtype in DTYPES:
        v = _inputs(5, 264, dtype, "token", True, True)
        v["res"][0] = 0
        v["y"][0] = 0
        v["y"][1] *= 2.0 ** -12
        v["res"][2] *= 100
        v["gate"][3], v["gate"][4] = 80.0, -80.0
        _check(moe, v, dtype, 1.0, 1.0, eps=1e-5)


def test_special_values_stay_in_their_rows(moe):
    v = _inputs(6, 264, torch.bfloat16, "token", True, True)
    v["y"][1, 3], v["res"][4, 9] = float("nan"), float("inf")
    d = {k: gpu(t) for k, t in v.items()}
    r, n, sp, sn = moe.moe_block_norm(d["res"], d["y"], gate=d["gate"], w_post=d["w_post"], w_pre=d["w_pre"])
    assert (~torch.isfinite(n.float())).any(1).tolist() == [False, True, False, False, True, False]
    assert torch.isnan(r.float()).all(1).tolist() == [False, True, False, False, False, False]


def test_update_in_place_equals_the_separate_one(moe):
    for T, H in ((5, 2048), (600, 264)):
        v = _inputs(T, H, torch.bfloat16, "element", False, True)
        d = {k: gpu(t) for k, t in v.items()}
        r, n, _, _ = moe.moe_block_norm(d["res"], d["y"], gate=d["gate"], w_pre=d["w_pre"], out_scale=0.5)
        res = d["res"].clone()
        r2, n2, _, _ = moe.moe_block_norm(res, d["y"], gate=d["gate"], w_pre=d["w_pre"], out_scale=0.5, r_out=res)
        assert r2 is res and torch.equal(r, res) and torch.equal(n, n2)


def test_weight_gradients_do_not_depend_on_timing(moe):
    v = _inputs(3000, 1032, torch.float32, "token", True, True)
    first = _check(moe, v, torch.float32, 1.0, 1.0)[2]
    for _ in range(3):
        again = _check(moe, v, torch.float32, 1.0, 1.0)[2]
        for p, q in zip(first, again):
            assert torch.equal(p, q)


def test_python_refusals(moe):
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(16, device="cuda")
    with pytest.raises(ValueError, match="without y"):
        moe.moe_block_norm(x)
    with pytest.raises(ValueError, match="float32"):
        moe.moe_block_norm(x, x, w_post=w.bfloat16())
    with pytest.raises(ValueError, match="shape"):
        moe.moe_block_norm(x, x, gate=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="bfloat16"):
        moe.moe_block_norm(x, x.half())
    with pytest.raises(ValueError, match="together"):
        moe.moe_block_norm_grad(x, None, x, w_pre=w, rstd_pre=w[:4])
    with pytest.raises(ValueError, match="rstd_post"):
        moe.moe_block_norm_grad(x, None, x, y=x, w_post=w)
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_block_norm_grad(x, x, x, y=x, w_pre=w, rstd_pre=w[:4].contiguous(),
                                ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
