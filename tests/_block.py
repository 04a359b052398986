"""Inputs and bounds shared by the GPU tests of the sort, norm and e4m3 operators."""
import numpy as np
import torch

# half a unit of rounding to each type, and the type's smallest step near zero
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SMALL = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
U32 = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def gpu(t):
    return None if t is None else t.cuda()


def within(got, ref, bound, name):
    """|got - ref| <= bound elementwise; NaN and infinities in the same places."""
    half = isinstance(got, torch.Tensor) and got.dtype == torch.float16
    got = f64(got) if isinstance(got, torch.Tensor) else np.asarray(got, dtype=np.float64)
    ref, bound = np.broadcast_to(ref, got.shape), np.broadcast_to(bound, got.shape)
    if half:
        # float16 ends at 65504 and rounds to infinity from 65520 on; where the
        # bound reaches that border, infinity is as right as the last value
        over = np.isfinite(ref) & (np.abs(ref) + bound >= 65520)
        assert np.all(np.abs(got[over]) >= 65504 - bound[over]), f"{name}: no overflow"
        got, ref = np.where(over, 0.0, got), np.where(over, 0.0, ref)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN elsewhere"
    assert np.array_equal(got[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)]), f"{name}: infinities"
    over = np.abs(got[fine] - ref[fine]) - bound[fine]
    worst = float(np.max(np.abs(got[fine] - ref[fine]) / np.maximum(bound[fine], 1e-300))) if over.size else 0.0
    assert not over.size or over.max() <= 0, f"{name}: {worst:.3g} times the bound"


def rounded(ref, dtype, err):
    """Bound of a value computed in f32 with error err and rounded to dtype once."""
    return err + UNIT[dtype] * (np.abs(ref) + err) + SMALL[dtype]


def permutation(gen, T, K, has_shared):
    pos = torch.randperm(T * K, generator=gen)
    if has_shared:
        pos = torch.cat([pos, T * K + torch.randperm(T, generator=gen)])
    return pos.int()
