"""The norm of many gradients and their clipping on the GPU against the oracle.

The squares are summed in 64 bits: the norm is the exact one rounded to f32, give or take
one more unit (2^-23 relative).  The scaled values are defined to the bit by the norm."""
import numpy as np
import pytest
import torch

from _block import DTYPES, f64, gpu, normal
from _gpu import flush, setup
from oracle import grad_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


def _scaled(g, norm, top):
    c = grad_norm.factor32(float(norm), top)
    return (g.cpu().float() * torch.tensor(c)).to(g.dtype)


def _same(a, b):
    a, b = a.cpu(), b.cpu()
    return torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)]) and torch.equal(torch.isnan(a), torch.isnan(b))


def _check(moe, grads, top):
    norm = moe.moe_grad_norm(grads)
    ref = grad_norm.norm([f64(g) for g in grads])
    assert norm.shape == (1,) and norm.dtype == torch.float32
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref, (float(norm), ref)
    out = [torch.full_like(g, 5.0) for g in grads]
    r = moe.moe_grad_clip(grads, norm, top, out=out)
    assert all(a is b for a, b in zip(r, out))
    for g, o in zip(grads, out):
        assert _same(o, _scaled(g, norm, top))
    return norm, out


@pytest.mark.parametrize("over", [0.5, 3.0])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [[1], [7], [8], [1000], [16384], [16385], [65537, 3, 0, 16, 1], [40000] * 5,
                                   [33] * 112, [5] * 113, list(range(300)), [3000001]])
def test_norm_and_clip(moe, sizes, dtype, over):
    flush(f"clip {len(sizes)} tensors of up to {max(sizes)} {dtype}")
    gen = torch.Generator().manual_seed(len(sizes))
    grads = [gpu(normal(gen, (n,), dtype, 0.1)) for n in sizes]
    _check(moe, grads, 0.1 * np.sqrt(sum(sizes)) / over)


def test_mixed_types_shapes_and_layouts(moe):
    gen = torch.Generator().manual_seed(0)
    grads = [gpu(normal(gen, s, t)) for s, t in (((30, 40), DTYPES[0]), ((3, 5, 7), DTYPES[1]), ((), DTYPES[2]),
                                                 ((0, 4), DTYPES[0]), ((513, 129), DTYPES[2]))]
    grads += [grads[0].t(), gpu(normal(gen, (2, 6, 5, 4), DTYPES[0])).to(memory_format=torch.channels_last)]
    norm = moe.moe_grad_norm(grads)
    ref = grad_norm.norm([f64(g) for g in grads])
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    grads = grads[:5] + [grads[5].clone(memory_format=torch.preserve_format), grads[6]]
    want = [_scaled(g, norm, 1.0) for g in grads]
    got = moe.moe_grad_clip(grads, norm, 1.0)
    for g, w, o in zip(grads, want, got):
        assert o is g and _same(g, w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (1, 1), (3, 3), (0, 1), (3, 0), (5, 2)])
def test_any_alignment(moe, shift_in, shift_out, dtype):
    """Pieces of one buffer at any place: nothing beside them is read into the norm or written."""
    gen = torch.Generator().manual_seed(1)
    n = [1, 2, 9, 33, 16384, 20001]
    for size in n:
        src = torch.full((size + 64,), 1e4, dtype=dtype, device="cuda")
        dst = torch.full((size + 64,), 3.0, dtype=dtype, device="cuda")
        g, o = src[16 + shift_in:16 + shift_in + size], dst[16 + shift_out:16 + shift_out + size]
        g.copy_(gpu(normal(gen, (size,), dtype)))
        norm = moe.moe_grad_norm([g])
        ref = grad_norm.norm([f64(g)])
        assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
        moe.moe_grad_clip([g], norm, ref / 2, out=[o])
        assert _same(o, _scaled(g, norm, ref / 2))
        assert (dst[:16 + shift_out] == 3).all() and (dst[16 + shift_out + size:] == 3).all()


def test_values_whose_squares_pass_f32(moe):
    g = torch.full((1000,), 1e30, dtype=torch.bfloat16, device="cuda")
    small = torch.full((1000,), 1e-30, device="cuda")
    for t in (g, small):
        _check(moe, [t], 1.0)
    g = torch.full((40000,), 3e38, device="cuda")  # a norm of 6e40: past f32, hence infinite
    norm = moe.moe_grad_norm([g])
    assert torch.isinf(norm).all() and not moe.moe_grad_clip([g], norm, 1.0)[0].any()


def test_not_finite(moe):
    a, b = torch.ones(100, device="cuda"), torch.ones(50, device="cuda")
    b[7] = float("inf")
    norm, out = moe.moe_grad_norm([a, b]), None
    assert torch.isinf(norm).all()
    out = moe.moe_grad_clip([a, b], norm, 1.0, out=[torch.empty_like(a), torch.empty_like(b)])
    assert not out[0].any() and torch.isnan(out[1][7]) and not out[1][:7].any()
    b[7] = float("nan")
    norm = moe.moe_grad_norm([a, b])
    assert torch.isnan(norm).all()
    moe.moe_grad_clip([a, b], norm, 1.0)
    assert torch.isnan(a).all() and torch.isnan(b).all()


def test_zeros_and_a_limit_of_zero(moe):
    z = torch.zeros(77, device="cuda")
    norm, _ = _check(moe, [z], 1.0)
    assert float(norm) == 0
    empty = torch.zeros(0, device="cuda")
    assert float(moe.moe_grad_norm([empty])) == 0
    assert moe.moe_grad_clip([empty], norm, 1.0)[0] is empty
    g = torch.ones(9, device="cuda")
    moe.moe_grad_clip([g], moe.moe_grad_norm([g]), 0.0)
    assert not g.any()


def test_in_place_and_repeated(moe):
    gen = torch.Generator().manual_seed(3)
    grads = [gpu(normal(gen, (n,), t)) for n, t in ((5000, DTYPES[0]), (40001, DTYPES[2]), (17, DTYPES[1]))]
    keep = [g.clone() for g in grads]
    norms = [moe.moe_grad_norm(grads) for _ in range(3)]
    assert all(torch.equal(n, norms[0]) for n in norms)
    moe.moe_grad_clip(grads, norms[0], 1e6)        # far below the limit: unchanged
    assert all(torch.equal(g, k) for g, k in zip(grads, keep))
    moe.moe_grad_clip(grads, norms[0], 2.0)
    for g, k in zip(grads, keep):
        assert torch.equal(g.cpu(), _scaled(k, norms[0], 2.0))


def test_python_refusals(moe):
    g = torch.zeros(8, 8, device="cuda")
    norm = torch.zeros(1, device="cuda")
    with pytest.raises(ValueError, match="gaps"):
        moe.moe_grad_norm([g[:, :4]])
    with pytest.raises(ValueError, match="gaps"):
        moe.moe_grad_norm([g[:1].expand(8, 8)])
    with pytest.raises(ValueError, match="float32"):
        moe.moe_grad_norm([g.double()])
    with pytest.raises(ValueError, match="on cuda:0, got cpu"):
        moe.moe_grad_norm([g, torch.zeros(4)])
    with pytest.raises(ValueError, match="out has 2"):
        moe.moe_grad_clip([g], norm, 1.0, out=[g, g])
    for o in (g.half(), g.t(), g[:4], g.cpu()):
        with pytest.raises(ValueError, match=r"out\[0\]"):
            moe.moe_grad_clip([g], norm, 1.0, out=[o])
    with pytest.raises(ValueError, match="shape"):
        moe.moe_grad_clip([g], torch.zeros((), device="cuda"), 1.0)
    with pytest.raises(moe.ops._lib.MoeError, match="max_norm"):
        moe.moe_grad_clip([g], norm, -1.0)
