"""The lists that moe_grad_norm and moe_grad_clip take: a call keeps the tensors that were
in the list when it began, whatever becomes of the list meanwhile."""
import threading
import time

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from _gpu import flush, setup

pytestmark = pytest.mark.gpu
N = 1 << 20


@pytest.fixture(scope="module")
def moe():
    return setup()


def test_a_list_emptied_while_the_output_is_allocated(moe):
    """A dispatch mode is Python code inside the call: what it drops from the list is still
    summed, and its memory is nobody else's yet."""
    flush("gradient list emptied during the call")
    grads, others = [torch.full((N,), 2.0, device="cuda") for _ in range(3)], []

    class Empties(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if grads and "empty" in str(func):
                grads.clear()
                others.extend(torch.full((N,), 7.0, device="cuda") for _ in range(3))
            return func(*args, **(kwargs or {}))

    with Empties():
        norm = moe.moe_grad_norm(grads)
    assert not grads and len(others) == 3
    ref = (3 * N * 4.0) ** 0.5
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    assert all((o == 7).all() for o in others)


def test_a_list_emptied_by_another_thread(moe):
    """A call that waits (here for the timing lock, which a reader of a long run holds) has the
    interpreter's lock given away: a list emptied meanwhile does not free the gradients."""
    from bit_block_quantized_nvfp4_amd import ops

    grads = [torch.full((N,), 2.0, device="cuda") for _ in range(3)]
    norm = moe.moe_grad_norm(grads)
    top = float(norm) / 2  # here: reading it waits for the device
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    torch.cuda._sleep(1000)
    ends[0].record()
    torch.cuda._sleep(100000)
    ends[1].record()
    torch.cuda.synchronize()
    cycles = int(100000 * 400 / max(ends[0].elapsed_time(ends[1]), 1e-2))
    flush(f"gradient list emptied by another thread, spin of {cycles} cycles")
    given = list(grads)
    got = []
    ops.timing_reset()
    ops.timing_enable(True)
    try:
        torch.cuda._sleep(cycles)
        small = moe.moe_grad_norm([norm])                     # its end is the spin's
        reader = threading.Thread(target=ops.timing_read)
        clip = threading.Thread(target=lambda: got.append(moe.moe_grad_clip(given, norm, top)))
        reader.start()
        time.sleep(0.05)                                      # the reader has the lock
        clip.start()
        time.sleep(0.05)                                      # the call waits for it
        grads.clear()
        given.clear()
        others = [torch.full((N,), 7.0, device="cuda") for _ in range(3)]
        reader.join()
        clip.join()
    finally:
        ops.timing_enable(False)
        ops.timing_reset()
    torch.cuda.synchronize()
    assert small.numel() == 1 and all((o == 7).all() for o in others)
    (scaled,) = got
    assert len(scaled) == 3 and all((s == 1).all() for s in scaled)


def test_the_result_is_a_list_of_the_scaled_tensors(moe):
    grads = (torch.full((5,), 2.0, device="cuda"), torch.full((7,), 2.0, device="cuda"))
    norm = moe.moe_grad_norm(list(grads))
    r = moe.moe_grad_clip(grads, norm, 1e6)
    assert isinstance(r, list) and all(a is b for a, b in zip(r, grads))
    out = [torch.empty_like(g) for g in grads]
    r = moe.moe_grad_clip(list(grads), norm, 1e6, out=out)
    assert isinstance(r, list) and r is not out and all(a is b for a, b in zip(r, out))
