"""The inputs of the GPU test of the e4m3 products' sums, checked on the host."""
import torch

from test_gpu_fp8_sums import _cancelling


def test_inputs_need_f32_sums_and_are_exact_in_them():
    x, w = _cancelling(torch.Generator().manual_seed(0), 2, 3, 400)
    p = (x[:, None] * w[None]).double()
    # multiples of 1/2, and no partial sum of a block of 128 in any order past 2^23
    assert (p * 2 == (p * 2).round()).all()
    assert all(p[..., b:b + 128].abs().sum(-1).max() < 2 ** 23 for b in range(0, 400, 128))
    assert all(torch.equal(v, v.to(torch.float8_e4m3fn).float()) for v in (x, w))
    # aligned to a run's largest product and cut 13 bits below, every run loses some
    run = p.abs().reshape(2, 3, -1, 8)
    unit = 2.0 ** (torch.floor(torch.log2(run.amax(-1))) - 13)
    assert (run.amin(-1) < unit).all()
