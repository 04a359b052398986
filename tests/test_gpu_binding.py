"""How the compiled marshalling behaves towards torch and Python: errors of the
library, other threads, outputs that torch can see, devices."""
import pytest
import torch

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
