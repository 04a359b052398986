"""The bf16 combine on both sides of its switch of kernels, and no slower than the
kernel of small batches where the other one's threads would stand idle."""
import pytest
import torch

from _gpu import flush, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


def _inputs(T, K, H):
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    y = torch.randn(T * K + T, H, generator=gen, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(T, K, generator=gen, device="cuda")
    pos = torch.cat([torch.randperm(T * K, generator=gen, device="cuda"),
                     T * K + torch.randperm(T, generator=gen, device="cuda")]).int()
    return y, w, pos, torch.randn(T, generator=gen, device="cuda")


def _few(y, w, pos, gate, a, b):
    """Tokens a .. b with the rows of their slots alone."""
    T, K = w.shape
    slots = torch.cat([pos[a * K:b * K], pos[T * K + a:T * K + b]])
    few = torch.where(slots >= 0, torch.arange(len(slots), device="cuda", dtype=torch.int32), slots)
    return y[slots.clamp_min(0).long()], w[a:b].contiguous(), few, gate[a:b].contiguous()


@pytest.mark.parametrize("T,K,H", [(6200, 10, 2048), (17600, 2, 2560), (60000, 2, 776), (3500, 4, 8192)])
def test_same_bits_for_many_rows(moe, T, K, H):
    flush(f"combine switch T={T} K={K} H={H}")
    y, w, pos, gate = _inputs(T, K, H)
    assert y.nbytes > 256 << 20
    pos[5::11] = -1
    y[100, 3], y[200, 5] = float("nan"), float("inf")
    out = moe.moe_combine_gated(y, w, pos, gate, K)
    for a in range(0, T, T // 7):
        b = min(T, a + 40)
        part = moe.moe_combine_gated(*_few(y, w, pos, gate, a, b), K)
        assert torch.equal(part.view(torch.int16), out[a:b].view(torch.int16))


def _us(f):
    for _ in range(3):
        f()
    best = float("inf")
    for _ in range(5):
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    return best


def test_a_row_past_the_switch_width_costs_what_its_bytes_cost(moe):
    """H = 2056 has 257 chunks of 16 bytes: a grid that gives such a row 512 threads
    took 39.6 us where H = 2048 takes 27.5 us (140 MB, K = 10)."""
    K, us = 10, {}
    for H in (2048, 2056):
        T = 140 * 2 ** 20 // ((K + 1) * H * 2)
        y, w, pos, _ = _inputs(T, K, H)
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        us[H] = _us(lambda: moe.moe_combine(y, w, pos, K, True, out=out))
    flush(f"combine 140 MB: {us}")
    assert us[2056] < 1.25 * us[2048]
