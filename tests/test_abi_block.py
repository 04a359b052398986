"""Refusals of the token sort, block norm and e4m3 entry points: reported on the
host, without a GPU, before anything is enqueued."""
import ctypes

import pytest
import torch

from _libutil import ensure_built

BF, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from bit_block_quantized_nvfp4_amd import _lib

    return _lib


@pytest.fixture(scope="module")
def lib(L):
    return L.lib()


P = ctypes.c_void_p(64)
ODD = ctypes.c_void_p(72)


def _is(L, lib, rc, status, text):
    assert rc == status, (rc, lib.moe_last_error())
    assert text in lib.moe_last_error(), lib.moe_last_error()


def test_sort_refusals(L, lib):
    calls = {
        "dispatch": lambda x=P, pos=P, T=4, K=2, H=16, sh=0, dt=BF, o=P: lib.moe_dispatch(x, pos, T, K, H, sh, dt, o, None),
        "dispatch_grad": lambda x=P, pos=P, T=4, K=2, H=16, sh=0, dt=BF, o=P: lib.moe_dispatch_grad(x, pos, T, K, H, sh, dt, o, None),
        "combine_typed": lambda x=P, pos=P, T=4, K=2, H=16, sh=0, dt=BF, o=P, g=None: lib.moe_combine_typed(x, P, pos, g, T, K, H, sh, dt, o, None),
        "combine_grad": lambda x=P, pos=P, T=4, K=2, H=16, sh=0, dt=BF, o=P, g=None, dg=None: lib.moe_combine_grad(x, P, P, pos, g, T, K, H, sh, dt, o, P, dg, None),
    }
    for name, f in calls.items():
        _is(L, lib, f(x=None), L.MOE_EINVAL, b"null")
        _is(L, lib, f(pos=None), L.MOE_EINVAL, b"null")
        _is(L, lib, f(o=None), L.MOE_EINVAL, b"null")
        _is(L, lib, f(T=0), L.MOE_EINVAL, b"T >= 1")
        _is(L, lib, f(K=0), L.MOE_EINVAL, b"K")
        _is(L, lib, f(K=33), L.MOE_EINVAL, b"K")
        _is(L, lib, f(H=12), L.MOE_EINVAL, b"multiple of 8")
        _is(L, lib, f(H=65544), L.MOE_EINVAL, b"65536")
        _is(L, lib, f(sh=2), L.MOE_EINVAL, b"has_shared")
        _is(L, lib, f(T=1 << 30, K=2), L.MOE_EINVAL, b"T")
        _is(L, lib, f(dt=3), L.MOE_EUNSUPPORTED, b"dtype")
        _is(L, lib, f(x=ODD), L.MOE_EINVAL, b"aligned")
        _is(L, lib, f(o=ODD), L.MOE_EINVAL, b"aligned")
        assert name.encode() in lib.moe_last_error()
    _is(L, lib, calls["combine_typed"](g=P), L.MOE_EINVAL, b"has_shared")
    _is(L, lib, calls["combine_grad"](g=P, dg=P), L.MOE_EINVAL, b"has_shared")
    _is(L, lib, calls["combine_grad"](g=P, sh=1), L.MOE_EINVAL, b"together")
    _is(L, lib, calls["combine_grad"](dg=P, sh=1), L.MOE_EINVAL, b"together")
    tg = lib.moe_route_topk_grad
    _is(L, lib, tg(None, P, P, 4, 8, 2, P, None), L.MOE_EINVAL, b"null")
    _is(L, lib, tg(P, P, P, 4, 8, 9, P, None), L.MOE_EINVAL, b"K <= min")
    _is(L, lib, tg(P, P, P, 4, 1025, 2, P, None), L.MOE_EINVAL, b"1024")


def test_norm_refusals(L, lib):
    def f(res=P, y=P, gate=None, kind=0, wpo=P, wpr=P, eps=1e-6, T=4, H=16, dt=BF, r=P, n=P, spo=P, spr=P):
        return lib.moe_block_norm(res, y, gate, kind, wpo, wpr, 1.0, 1.0, eps, T, H, dt, r, n, spo, spr, None)

    E = L.MOE_EINVAL
    _is(L, lib, f(res=None), E, b"null")
    _is(L, lib, f(T=0), E, b"T")
    _is(L, lib, f(H=20), E, b"multiple of 8")
    _is(L, lib, f(H=8200), E, b"8192")
    _is(L, lib, f(dt=7), L.MOE_EUNSUPPORTED, b"dtype")
    _is(L, lib, f(kind=3), L.MOE_EUNSUPPORTED, b"gate_kind")
    _is(L, lib, f(kind=1), E, b"agree")
    _is(L, lib, f(gate=P), E, b"agree")
    _is(L, lib, f(y=None), E, b"without y")
    _is(L, lib, f(y=None, wpo=None, r=None, wpr=None, n=None, spo=None, spr=None), E, b"without y")
    _is(L, lib, f(r=None), E, b"r_out")
    _is(L, lib, f(n=None), E, b"together")
    _is(L, lib, f(wpr=None), E, b"together")
    _is(L, lib, f(wpo=None), E, b"statistics")
    _is(L, lib, f(eps=-1.0), E, b"eps")
    _is(L, lib, f(eps=float("nan")), E, b"eps")
    for k in ("res", "y", "wpo", "wpr", "r", "n"):
        _is(L, lib, f(**{k: ODD}), E, b"aligned")
    _is(L, lib, f(gate=ODD, kind=2), E, b"aligned")

    ws = lib.moe_block_norm_workspace_bytes
    assert ws(4, 20, 0) == 0 and ws(0, 16, 0) == 0 and ws(4, 16, 9) == 0
    need = ws(4, 16, 0)
    assert need > 0

    def g(dr=P, dn=P, r=P, y=P, gate=None, kind=0, wpo=P, wpr=P, spo=P, spr=P, T=4, H=16, dt=BF, dres=P, dy=P,
          dg=None, dpo=P, dpr=P, w=P, nb=need):
        return lib.moe_block_norm_grad(dr, dn, r, y, gate, kind, wpo, wpr, spo, spr, 1.0, 1.0, T, H, dt, dres, dy,
                                       dg, dpo, dpr, w, nb, None)

    _is(L, lib, g(dres=None), E, b"null")
    _is(L, lib, g(dr=None, dn=None), E, b"null")
    _is(L, lib, g(kind=1, gate=P), E, b"agree")
    _is(L, lib, g(dg=P), E, b"agree")
    _is(L, lib, g(y=None), E, b"without y")
    _is(L, lib, g(dy=None), E, b"dy")
    for k in ("dn", "r", "spr", "dpr", "wpr"):
        _is(L, lib, g(**{k: None}), E, b"together")
    for k in ("spo", "dpo", "wpo"):
        _is(L, lib, g(**{k: None}), E, b"together")
    for k in ("dr", "dn", "r", "y", "wpo", "wpr", "dres", "dy", "w"):
        _is(L, lib, g(**{k: ODD}), E, b"aligned")
    _is(L, lib, g(w=None), L.MOE_EWORKSPACE, b"workspace")
    _is(L, lib, g(nb=need - 1), L.MOE_EWORKSPACE, b"workspace")


def test_fp8_refusals(L, lib):
    E = L.MOE_EINVAL
    q = lib.moe_fp8_quant
    _is(L, lib, q(None, 4, 128, BF, P, P, None), E, b"null")
    _is(L, lib, q(P, 4, 120, BF, P, P, None), E, b"multiple of 16")
    _is(L, lib, q(P, 0, 128, BF, P, P, None), E, b"T")
    _is(L, lib, q(P, 4, 65552, BF, P, P, None), E, b"65536")
    _is(L, lib, q(P, 4, 128, 5, P, P, None), L.MOE_EUNSUPPORTED, b"dtype")
    _is(L, lib, q(ODD, 4, 128, BF, P, P, None), E, b"aligned")
    wsb = lib.moe_fp8_linear_workspace_bytes
    assert wsb(16, 16, 128) == 0 and wsb(17, 16, 100) == 0 and wsb(17, 12, 144) == 0
    assert wsb(17, 16, 144) >= 17 * 256 + 17 * 2 * 4
    need = wsb(17, 16, 256)

    def f(codes=64, scales=64, N=16, K=256, x=P, T=17, dt=BF, o=P, ws=P, nb=need, M=True):
        m = L.MoeFp8Matrix(codes, scales, N, K)
        return lib.moe_fp8_linear(ctypes.byref(m) if M else None, x, T, dt, o, ws, nb, None)

    _is(L, lib, f(M=False), E, b"null")
    _is(L, lib, f(x=None), E, b"null")
    _is(L, lib, f(o=None), E, b"null")
    _is(L, lib, f(codes=0), E, b"weight pointer")
    _is(L, lib, f(scales=0), E, b"weight pointer")
    _is(L, lib, f(N=12), E, b"multiple of 8")
    _is(L, lib, f(K=250), E, b"multiple of 16")
    _is(L, lib, f(T=0), E, b"T")
    _is(L, lib, f(dt=4), L.MOE_EUNSUPPORTED, b"dtype")
    _is(L, lib, f(codes=72), E, b"aligned")
    _is(L, lib, f(x=ODD), E, b"aligned")
    _is(L, lib, f(o=ODD), E, b"aligned")
    _is(L, lib, f(ws=None), L.MOE_EWORKSPACE, b"workspace")
    _is(L, lib, f(nb=need - 1), L.MOE_EWORKSPACE, b"workspace")

    wse = lib.moe_fp8_expert_ffn_workspace_bytes
    assert wse(4, 2, 200, 128, 0) == 0 and wse(4, 33, 256, 128, 0) == 0 and wse(4, 2, 256, 128, 2) == 0
    need2 = wse(40, 2, 256, 128, 1)
    assert need2 >= 40 * 256 + (40 * 3) * 128

    def e(gu=64, gus=64, dn=64, dns=64, En=8, H=256, I=128, sh=1, x=P, T=40, K=2, o=P, off=P, ss=P, gr=P, ws=P,
          nb=need2):
        W = L.MoeFp8Weights(gu, gus, dn, dns, En, H, I, sh)
        return lib.moe_fp8_expert_ffn(ctypes.byref(W), x, T, K, off, ss, gr, o, ws, nb, None)

    for k in ("x", "o", "off", "ss", "gr"):
        _is(L, lib, e(**{k: None}), E, b"null")
    for k in ("gu", "gus", "dn", "dns"):
        _is(L, lib, e(**{k: 0}), E, b"weight pointer")
    _is(L, lib, e(H=192), E, b"multiples of 128")
    _is(L, lib, e(I=64), E, b"multiples of 128")
    _is(L, lib, e(H=8320), E, b"8192")
    _is(L, lib, e(K=9), E, b"K")
    _is(L, lib, e(sh=2), E, b"has_shared")
    _is(L, lib, e(gu=72), E, b"aligned")
    _is(L, lib, e(x=ODD), E, b"aligned")
    _is(L, lib, e(ws=None), L.MOE_EWORKSPACE, b"workspace")
    _is(L, lib, e(nb=need2 - 1), L.MOE_EWORKSPACE, b"workspace")


def test_python_entry_points_refuse_host_tensors(L):
    import bit_block_quantized_nvfp4_amd as moe

    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    pos = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_dispatch(x, pos, 2, False)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_block_norm(x, x)
    with pytest.raises(ValueError, match="device tensor"):
        moe.moe_fp8_quant(x)


def test_matrix_layout_on_the_host():
    """from_float and transposed keep the blocks: exact for representable values."""
    import bit_block_quantized_nvfp4_amd as moe

    g = torch.Generator().manual_seed(0)
    N, K = 264, 144
    # up to four significant bits each, and 448 = 14 * 32 in every block: e4m3 holds them
    w = torch.randint(-8, 9, (N, K), generator=g).float() * 32
    w[::128, ::128] = 448.0
    w[256:, 128:] *= 0.25
    w[256, 128] = 112.0
    M = moe.FP8Matrix.from_float(w)
    s = M.scales.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    assert M.scales.shape == (3, 2) and torch.equal(M.codes.float() * s, w)
    t = M.transposed()
    assert torch.equal(t.codes.float(), M.codes.float().t()) and torch.equal(t.scales, M.scales.t())
    zero = moe.FP8Matrix.from_float(torch.zeros(16, 16))
    assert torch.equal(zero.codes.float(), torch.zeros(16, 16))
