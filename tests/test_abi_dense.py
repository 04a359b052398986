"""Refusals of the dense block, 8-bit integer and gradient norm entry points: reported on
the host, without a GPU, before anything is enqueued."""
import ctypes

import pytest
import torch

from _libutil import ensure_built

BF, F16, F32 = 0, 1, 2
P = ctypes.c_void_p(64)
ODD = ctypes.c_void_p(72)


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from bit_block_quantized_nvfp4_amd import _lib

    return _lib


@pytest.fixture(scope="module")
def lib(L):
    return L.lib()


def _is(L, rc, status, text):
    msg = L.lib().moe_last_error()
    assert rc == status and text in msg, (rc, msg)


def test_dense_refusals(L, lib):
    E = L.MOE_EINVAL
    fb, gb = lib.moe_dense_ffn_workspace_bytes, lib.moe_dense_ffn_grad_workspace_bytes
    for b in (fb, gb):
        assert b(4, 12, 16) == 0 and b(0, 16, 16) == 0 and b(4, 16, 65544) == 0 and b(4, 16, 24) > 0
    assert fb(1000, 512, 512) >= 1000 * 512 * 2 and gb(1000, 512, 512) >= 1000 * 512 * 6

    def f(gu=64, dn=64, H=64, I=32, dt=BF, x=P, T=4, y=P, k=None, ws=P, nb=None, W=True):
        w = L.MoeDenseWeights(gu, dn, H, I, dt)
        return lib.moe_dense_ffn(ctypes.byref(w) if W else None, x, T, y, k, ws, fb(T, H, I) if nb is None else nb, None)

    def g(gu=64, dn=64, H=64, I=32, dt=F16, dy=P, x=P, k=P, T=4, dx=P, dg=P, dd=P, ws=P, nb=None, W=True):
        w = L.MoeDenseWeights(gu, dn, H, I, dt)
        return lib.moe_dense_ffn_grad(ctypes.byref(w) if W else None, dy, x, k, T, dx, dg, dd, ws,
                                      gb(T, H, I) if nb is None else nb, None)

    for c in (f, g):
        _is(L, c(W=False), E, b"null")
        _is(L, c(x=None), E, b"null")
        _is(L, c(gu=0), E, b"weight pointer")
        _is(L, c(dn=0), E, b"weight pointer")
        _is(L, c(dt=F32), L.MOE_EUNSUPPORTED, b"dtype")
        _is(L, c(T=0), E, b"1 <= T")
        _is(L, c(H=12), E, b"multiples of 8")
        _is(L, c(I=4), E, b"multiples of 8")
        _is(L, c(H=65544), E, b"65536")
        _is(L, c(gu=72), E, b"aligned")
        _is(L, c(dn=72), E, b"aligned")
        _is(L, c(x=ODD), E, b"aligned")
        _is(L, c(ws=ODD), E, b"aligned")
        _is(L, c(ws=None), L.MOE_EWORKSPACE, b"workspace")
        _is(L, c(nb=63), L.MOE_EWORKSPACE, b"workspace")
        _is(L, c(T=1 << 30, H=65536, I=65536), E, b"2^32 threads")
    for c in (f, g):
        _is(L, c(T=(1 << 30) + 1, H=8, I=8), E, b"2^30")
    _is(L, f(y=None), E, b"null")
    _is(L, f(y=ODD), E, b"aligned")
    _is(L, f(k=ODD), E, b"aligned")
    for k in ("dy", "k", "dx", "dg", "dd"):
        _is(L, g(**{k: None}), E, b"null")
        _is(L, g(**{k: ODD}), E, b"aligned")


def test_int8_refusals(L, lib):
    E = L.MOE_EINVAL
    q = lib.moe_int8_quant
    _is(L, q(None, 4, 64, BF, P, P, None), E, b"null")
    _is(L, q(P, 4, 64, BF, P, None, None), E, b"null")
    _is(L, q(P, 4, 72, BF, P, P, None), E, b"multiple of 16")
    _is(L, q(P, 0, 64, BF, P, P, None), E, b"T >= 1")
    _is(L, q(P, 4, 65552, BF, P, P, None), E, b"65536")
    _is(L, q(P, 4, 64, 3, P, P, None), L.MOE_EUNSUPPORTED, b"dtype")
    _is(L, q(ODD, 4, 64, BF, P, P, None), E, b"aligned")
    _is(L, q(P, 4, 64, BF, ODD, P, None), E, b"aligned")
    _is(L, q(P, 1 << 24, 64, BF, P, P, None), E, b"2^32 threads")
    _is(L, q(P, 1 << 22, 8208, BF, P, P, None), E, b"2^32 threads")
    wsb = lib.moe_int8_linear_workspace_bytes
    assert wsb(100, 16, 72) == 0 and wsb(100, 12, 64) == 0 and wsb(0, 16, 64) == 0 and wsb(100, 131080, 64) == 0
    assert wsb(100, 16, 64) >= 100 * 64 + 400

    def f(codes=64, scales=64, N=32, K=64, x=P, T=100, dt=BF, gated=0, o=P, ws=P, nb=None, M=True):
        m = L.MoeInt8Matrix(codes, scales, N, K)
        return lib.moe_int8_linear(ctypes.byref(m) if M else None, x, T, dt, gated, o, ws,
                                   wsb(T, N, K) if nb is None else nb, None)

    _is(L, f(M=False), E, b"null")
    _is(L, f(x=None), E, b"null")
    _is(L, f(o=None), E, b"null")
    _is(L, f(codes=0), E, b"weight pointer")
    _is(L, f(scales=0), E, b"weight pointer")
    _is(L, f(N=12), E, b"multiple of 8")
    _is(L, f(N=24, gated=1), E, b"gated: 16")
    _is(L, f(gated=2), E, b"gated")
    _is(L, f(K=72), E, b"multiple of 16")
    _is(L, f(T=0), E, b"T >= 1")
    _is(L, f(dt=9), L.MOE_EUNSUPPORTED, b"dtype")
    _is(L, f(codes=72), E, b"aligned")
    for k in ("x", "o", "ws"):
        _is(L, f(**{k: ODD}), E, b"aligned")
    _is(L, f(ws=None), L.MOE_EWORKSPACE, b"workspace")
    _is(L, f(nb=wsb(100, 32, 64) - 1), L.MOE_EWORKSPACE, b"workspace")
    _is(L, f(T=1 << 24), E, b"2^32 threads")


def test_gradient_list_refusals(L, lib):
    E = L.MOE_EINVAL
    wsb = lib.moe_grad_norm_workspace_bytes
    assert wsb(0) == 0 and wsb((1 << 20) + 1) == 0 and wsb(1) > 0

    def tensors(*items):
        return (L.MoeGradTensor * len(items))(*[L.MoeGradTensor(*i) for i in items])

    good = (64, 64, 10, BF)
    calls = {
        "norm": lambda t, n=None, norm=P, ws=P, nb=1 << 30: lib.moe_grad_norm(t, len(t) if n is None else n, norm, ws, nb, None),
        "clip": lambda t, n=None, norm=P, top=1.0: lib.moe_grad_clip(t, len(t) if n is None else n, norm, top, None),
    }
    for name, f in calls.items():
        _is(L, f(None, 1), E, b"null")
        _is(L, f(tensors(good), norm=None), E, b"null")
        _is(L, f(tensors(good), n=0), E, b"between 1 and 2^20")
        _is(L, f(tensors(good), n=(1 << 20) + 1), E, b"between 1 and 2^20")
        _is(L, f(tensors(good, (64, 64, 10, 3))), L.MOE_EUNSUPPORTED, b"tensor 1: unknown dtype")
        _is(L, f(tensors(good, (64, 64, -1, BF))), E, b"tensor 1: need 0 <= n")
        _is(L, f(tensors(good, (64, 64, (1 << 37) + 1, BF))), E, b"2^37")
        _is(L, f(tensors(good, good, (0, 64, 10, BF))), E, b"tensor 2: null pointer")
        _is(L, f(tensors((65, 65, 10, BF))), E, b"not aligned")
        _is(L, f(tensors((66, 66, 10, F32))), E, b"not aligned")
        assert b"moe_grad_" + name.encode() in lib.moe_last_error()
    clip = calls["clip"]
    _is(L, clip(tensors((64, 0, 10, BF))), E, b"null pointer")
    _is(L, clip(tensors((64, 65, 10, BF))), E, b"not aligned")
    for top in (-1.0, float("inf"), float("nan")):
        _is(L, clip(tensors(good), top=top), E, b"max_norm")
    _is(L, clip(tensors(good, good)), E, b"overlap")
    _is(L, clip(tensors((64, 100, 4, F32), (64, 64, 10, BF), (64, 84, 9, BF))), E, b"overlap")
    for other in ((64, 1000, 10, BF), (60, 1000, 4, BF), (83 & ~1, 1000, 2, BF)):
        _is(L, clip(tensors((2000, 64, 10, BF), other)), E, b"not its own")
    _is(L, clip(tensors((64, 66, 10, BF))), E, b"not its own")
    norm = calls["norm"]
    _is(L, norm(tensors(good), ws=None), L.MOE_EWORKSPACE, b"workspace")
    _is(L, norm(tensors(good), nb=wsb(1) - 1), L.MOE_EWORKSPACE, b"workspace")
    _is(L, norm(tensors(good), ws=ctypes.c_void_p(68)), L.MOE_EWORKSPACE, b"aligned to 8")


def test_python_entry_points_refuse_host_tensors_and_other_lists(L):
    import bit_block_quantized_nvfp4_amd as moe

    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    W = moe.DenseWeights(torch.zeros(32, 16, dtype=torch.bfloat16), torch.zeros(16, 16, dtype=torch.bfloat16))
    for call in (lambda: moe.moe_dense_ffn(W, x), lambda: moe.moe_dense_ffn_grad(W, x, x, x),
                 lambda: moe.moe_int8_quant(x), lambda: moe.moe_grad_norm([x]),
                 lambda: moe.moe_int8_linear(moe.Int8Matrix.from_float(torch.zeros(16, 16)), x),
                 lambda: moe.moe_grad_clip([x], torch.zeros(1), 1.0)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="empty"):
        moe.moe_grad_norm([])
    for bad in (x, iter([x]), None):
        with pytest.raises(ValueError, match="list or tuple"):
            moe.moe_grad_norm(bad)
    with pytest.raises(ValueError, match=r"grads\[0\] must be a tensor|must be a tensor"):
        moe.moe_grad_norm([1.0])


def test_int8_matrix_layout_on_the_host():
    """from_float: exact where a row's values are multiples of its largest / 127."""
    import bit_block_quantized_nvfp4_amd as moe

    gen = torch.Generator().manual_seed(0)
    codes = torch.randint(-127, 128, (24, 32), generator=gen)
    codes[:, 0] = 127
    scale = 2.0 ** torch.randint(-6, 6, (24,), generator=gen)
    M = moe.Int8Matrix.from_float(codes * scale[:, None])
    assert M.codes.dtype == torch.int8 and torch.equal(M.codes.long(), codes) and torch.equal(M.scales, scale)
    zero = moe.Int8Matrix.from_float(torch.zeros(8, 16))
    assert not zero.codes.any() and torch.isfinite(zero.scales).all()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are none; without a device nothing is launched")
def test_calls_within_the_limits_are_accepted(L, lib):
    """They get past every check, to the device that is missing here."""
    big = 1 << 60
    w = L.MoeDenseWeights(64, 64, 64, 64, BF)
    m = L.MoeInt8Matrix(64, 64, 131072, 65536)
    side = (L.MoeGradTensor * 4)(*[L.MoeGradTensor(*t) for t in ((64, 64, 10, BF), (64, 84, 0, BF), (128, 84, 9, BF), (600, 102, 1, F16))])
    apart = (L.MoeGradTensor * 3)(*[L.MoeGradTensor(*t) for t in ((64, 1084, 10, BF), (84, 1000, 10, BF), (64, 2000, 10, BF))])
    calls = [lambda: lib.moe_dense_ffn(ctypes.byref(w), P, 1 << 27, P, P, P, big, None),
             lambda: lib.moe_dense_ffn_grad(ctypes.byref(w), P, P, P, 1 << 27, P, P, P, P, big, None),
             lambda: lib.moe_int8_linear(ctypes.byref(m), P, (1 << 22) - 1, BF, 1, P, P, big, None),
             lambda: lib.moe_int8_quant(P, (1 << 24) - 1, 64, F32, P, P, None),
             lambda: lib.moe_grad_clip(side, 4, P, 0.0, None), lambda: lib.moe_grad_clip(apart, 3, P, 0.0, None),
             lambda: lib.moe_grad_norm(side, 4, P, P, big, None)]
    for f in calls:
        assert f() in (L.MOE_EHIP, L.MOE_EUNSUPPORTED), lib.moe_last_error()
