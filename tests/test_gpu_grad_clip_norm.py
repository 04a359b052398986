"""moe_grad_clip reads the norm while it writes: an output that holds it is refused, in
place or beside, before anything is launched."""
import pytest
import torch

from _gpu import flush, setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [0, 32, 63])
def test_an_output_that_holds_the_norm_is_refused(moe, at, dtype):
    flush(f"norm in an output, place {at} {dtype}")
    buf = torch.full((64,), 3.0, device="cuda")
    norm, tensor = buf[at:at + 1], buf.view(dtype)
    other = torch.ones(9, device="cuda")
    with pytest.raises(ValueError, match=r"grads\[1\] holds the norm"):
        moe.moe_grad_clip([other, tensor], norm, 1.0)
    with pytest.raises(ValueError, match=r"out\[0\] holds the norm"):
        moe.moe_grad_clip([torch.ones_like(tensor), other], norm, 1.0, out=[tensor, torch.empty_like(other)])
    assert (buf == 3).all() and (other == 1).all()


def test_outputs_beside_the_norm_and_a_gradient_that_is_one(moe):
    flush("outputs beside the norm")
    buf = torch.full((64,), 2.0, device="cuda")
    norm = buf[32:33]
    moe.moe_grad_clip([buf[:32], buf[33:], buf[40:40]], norm, 1.0)  # c = 1 / (2 + 1e-6)
    c = float(torch.tensor(1.0) / (torch.tensor(2.0) + torch.tensor(1e-6)))
    assert float(norm) == 2 and (buf[:32] == 2 * c).all() and (buf[33:] == 2 * c).all()
    out = torch.empty(64, device="cuda")
    before = buf.clone()
    moe.moe_grad_clip([buf], norm, 1.0, out=[out])  # read only: the norm among the gradients
    assert torch.equal(buf, before) and torch.equal(out, buf * torch.tensor(c, device="cuda"))
