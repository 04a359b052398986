"""How the compiled marshalling behaves towards torch and Python: errors of the
library, other threads, outputs that torch can see, devices."""
import threading
import time

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from _gpu import flush, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


def test_an_empty_batch_is_the_librarys_error(moe):
    err = moe.ops._lib.MoeError
    y, w = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 2, device="cuda")
    pos, gate = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda")
    for call in (lambda: moe.moe_combine(y, w, pos, 2, False), lambda: moe.moe_combine_gated(y, w, pos, gate, 2),
                 lambda: moe.moe_dispatch(y, pos, 2, False), lambda: moe.moe_dispatch_grad(y, pos, 2, True),
                 lambda: moe.moe_combine_grad(y, y, w, pos, 2, False), lambda: moe.moe_fp8_quant(y),
                 lambda: moe.moe_block_norm(y, y), lambda: moe.moe_route_topk_grad(w.int(), w, w, 4)):
        with pytest.raises(err) as e:
            call()
        assert e.value.status == moe.ops._lib.MOE_EINVAL


def test_a_call_that_waits_lets_other_threads_run(moe):
    """moe_timing_read holds the timing lock until the work before it is done; a call
    that waits for that lock must not hold the interpreter's."""
    x = torch.randn(8, 64, device="cuda").bfloat16()
    pos = torch.arange(16, dtype=torch.int32, device="cuda")
    y, w = moe.moe_dispatch(x, pos, 2, False), torch.rand(8, 2, device="cuda")
    want = moe.moe_combine(y, w, pos, 2, False)
    # a spin of about 0.4 s, by a short one's measure
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    torch.cuda._sleep(1000)
    ends[0].record()
    torch.cuda._sleep(100000)
    ends[1].record()
    torch.cuda.synchronize()
    cycles = int(100000 * 400 / max(ends[0].elapsed_time(ends[1]), 1e-2))
    flush(f"spin of {cycles} cycles")

    from bit_block_quantized_nvfp4_amd import ops
    stop, ticks = threading.Event(), []

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    ops.timing_reset()
    ops.timing_enable(True)
    try:
        torch.cuda._sleep(cycles)
        moe.moe_combine(y, w, pos, 2, False)          # its end is the spin's
        reader, ticker = threading.Thread(target=ops.timing_read), threading.Thread(target=tick)
        ticker.start()
        reader.start()
        time.sleep(0.05)                              # the reader has the lock
        a = time.perf_counter()
        out = moe.moe_combine(y, w, pos, 2, False)
        b = time.perf_counter()
        stop.set()
        reader.join()
        ticker.join()
    finally:
        stop.set()
        ops.timing_enable(False)
        ops.timing_reset()
    torch.cuda.synchronize()
    during = sum(a < t < b for t in ticks)
    flush(f"the call took {b - a:.3f} s, {during} ticks meanwhile")
    assert torch.equal(out, want)
    assert b - a > 0.1 and during >= 10


def test_torch_sees_new_outputs(moe):
    """Through torch's dispatcher: a dispatch mode meets them, and where deterministic
    algorithms are asked for, rows that a call leaves as they were are filled."""
    T, K, H = 6, 2, 64
    x = torch.randn(T, H, device="cuda").bfloat16()
    pos = torch.arange(T * K, dtype=torch.int32, device="cuda")
    y, w = moe.moe_dispatch(x, pos, K, False), torch.rand(T, K, device="cuda")

    class Seen(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            names.append(str(func))
            return func(*args, **(kwargs or {}))

    names = []
    with Seen():
        out = moe.moe_combine(y, w, pos, K, False)
    assert any("empty" in n for n in names), names
    assert torch.equal(out, moe.moe_combine(y, w, pos, K, False))

    pos[3] = -1
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        xs = moe.moe_dispatch(x, pos, K, False)
    finally:
        torch.use_deterministic_algorithms(before)
    assert torch.isnan(xs[3]).all() and not torch.isnan(xs[[0, 1, 2, 4]]).any()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_tensors_of_another_device(moe):
    """Run where the tensors are, on that device's current stream; the current device stays."""
    T, K, H = 9, 2, 264
    x, w, pos = torch.randn(T, H), torch.rand(T, K), torch.randperm(T * K).int()
    got = []
    for dev in ("cuda:0", "cuda:1"):
        stream = torch.cuda.Stream(dev)
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            a = [t.to(dev) for t in (x, w, pos)]
        stream.synchronize()
        torch.cuda.set_device(0)
        xs = moe.moe_dispatch(a[0], a[2], K, False)
        got.append(moe.moe_combine(xs, a[1], a[2], K, False))
        assert torch.cuda.current_device() == 0 and got[-1].device == torch.device(dev)
        torch.cuda.synchronize(dev)
    assert torch.equal(got[0].cpu(), got[1].cpu())


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two devices")
def test_layer_on_another_device(moe):
    """All of a layer's kernels on one stream of its tensors' device, in both forms."""
    import numpy as np

    from workloads import workload_for

    wl = workload_for("tiny")
    got = []
    for dev in ("cuda:0", "cuda:1"):
        W = moe.NVFP4Weights.from_bank(wl.weights, dev)
        x = torch.from_numpy(wl.x_bf16.view(np.int16)).to(dev).view(torch.bfloat16)
        logits = torch.from_numpy(wl.logits).to(dev)
        torch.cuda.synchronize(dev)
        for fused in (False, True):
            got.append(moe.moe_layer(W, x, logits, wl.K, fused=fused)["out"])
            torch.cuda.synchronize(dev)
    assert all(torch.equal(got[0].cpu(), g.cpu()) for g in got[1:])
