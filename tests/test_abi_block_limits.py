"""Sizes past what int32 positions and a HIP launch hold are refused on the host;
the largest sizes below are not (they end at the missing device here, or are not
launched at all)."""
import ctypes

import pytest
import torch

from _libutil import ensure_built

P = ctypes.c_void_p(64)
BF, F32 = 0, 2


@pytest.fixture(scope="module")
def L():
    ensure_built()
    from bit_block_quantized_nvfp4_amd import _lib

    return _lib


def _refused(L, rc, text):
    msg = L.lib().moe_last_error()
    assert rc == L.MOE_EINVAL and text in msg, (rc, msg)


@pytest.mark.parametrize("dt", [BF, F32])
def test_shared_positions_fit_int32(L, dt):
    """T*K = 2^30 alone is within the limits; with as many shared slots positions would reach 2^31."""
    lib, T = L.lib(), 1 << 30
    _refused(L, lib.moe_dispatch(P, P, T, 1, 8, 1, dt, P, None), b"2^31")
    _refused(L, lib.moe_dispatch_grad(P, P, T, 1, 8, 1, dt, P, None), b"2^31")
    _refused(L, lib.moe_combine_typed(P, P, P, None, T, 1, 8, 1, dt, P, None), b"2^31")
    _refused(L, lib.moe_combine_grad(P, P, P, P, None, T, 1, 8, 1, dt, P, P, None, None), b"2^31")
    _refused(L, lib.moe_combine(P, P, P, T, 1, 8, 1, P, None), b"2^31")
    _refused(L, lib.moe_combine_gated(P, P, P, P, T, 1, 8, P, None), b"2^31")
    _refused(L, lib.moe_permute(P, T, 8, 1, 1, P, P, P, P, P, None, 0, None), b"2^31")
    _refused(L, lib.moe_route_permute(P, T, 8, 1, 1, P, P, P, P, P, P, P, None, 0, None), b"2^31")


def test_grids_stay_below_2_32_threads(L):
    lib = L.lib()
    _refused(L, lib.moe_combine_grad(P, P, P, P, None, 1 << 25, 1, 8, 1, BF, P, P, None, None), b"2^32 threads")
    _refused(L, lib.moe_route_topk_grad(P, P, P, 1 << 26, 8, 2, P, None), b"2^32 threads")
    _refused(L, lib.moe_dispatch(P, P, 1 << 24, 1, 2048, 0, BF, P, None), b"2^32 threads")
    _refused(L, lib.moe_dispatch_grad(P, P, 1 << 20, 1, 65536, 0, BF, P, None), b"2^32 threads")
    _refused(L, lib.moe_combine_typed(P, P, P, None, 1 << 23, 1, 2048, 0, F32, P, None), b"2^32 threads")
    _refused(L, lib.moe_combine(P, P, P, 1 << 24, 1, 2048, 0, P, None), b"2^32 threads")
    _refused(L, lib.moe_block_norm(P, P, None, 0, P, P, 1.0, 1.0, 1e-6, 1 << 26, 8, BF, P, P, P, P, None), b"2^32 threads")
    _refused(L, lib.moe_block_norm(P, P, None, 0, P, P, 1.0, 1.0, 1e-6, 1 << 24, 2056, BF, P, P, P, P, None), b"2^32 threads")
    _refused(L, lib.moe_fp8_quant(P, 1 << 28, 16, BF, P, P, None), b"2^32 threads")
    m = L.MoeFp8Matrix(64, 64, 65536, 16)
    _refused(L, lib.moe_fp8_linear(ctypes.byref(m), P, 1 << 24, BF, P, P, 1 << 60, None), b"2^32 threads")
    W = L.MoeFp8Weights(64, 64, 64, 64, 8, 8192, 8192, 1)
    assert lib.moe_fp8_expert_ffn(ctypes.byref(W), P, 1 << 18, 8, P, P, P, P, None, 0, None) == L.MOE_EWORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are none; without a device nothing is launched")
def test_sizes_below_the_limits_are_accepted(L):
    """They get past every check of sizes, to the device that is missing here."""
    lib = L.lib()
    calls = [lambda: lib.moe_dispatch(P, P, 1 << 30, 1, 8, 0, BF, P, None),
             lambda: lib.moe_combine(P, P, P, (1 << 30) - 1, 1, 8, 1, P, None),
             lambda: lib.moe_combine_grad(P, P, P, P, None, (1 << 25) - 4, 1, 8, 1, BF, P, P, None, None),
             lambda: lib.moe_route_topk_grad(P, P, P, (1 << 26) - 4, 8, 2, P, None),
             lambda: lib.moe_block_norm(P, P, None, 0, P, P, 1.0, 1.0, 1e-6, (1 << 26) - 4, 8, BF, P, P, P, P, None),
             lambda: lib.moe_fp8_quant(P, (1 << 28) - 16, 16, BF, P, P, None)]
    for f in calls:
        assert f() in (L.MOE_EHIP, L.MOE_EUNSUPPORTED), lib.moe_last_error()
