"""The streaming experts (few tokens) with more than 16 rows in a group, which take
a second pass over the group's weights, and with ids outside the bank, in each
of their wave shapes: by the number of groups that may be active (16, 48) and, for
down, a short or a long intermediate."""
import pytest
import torch

from _block import gpu, normal
from _gpu import flush, setup
from test_gpu_fp8 import _bank, _check_experts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    return setup()


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("T,E,K,H,I", [(8, 4, 3, 256, 128), (6, 8, 8, 384, 640), (8, 32, 4, 256, 256),
                                       (12, 64, 6, 256, 128), (12, 60, 5, 128, 640), (9, 128, 10, 128, 1024)])
def test_long_groups_and_foreign_ids(moe, T, E, K, H, I, shared):
    flush(f"fp8 stream, long group T={T} E={E} K={K} H={H} I={I} shared={shared}")
    gen = torch.Generator().manual_seed(T + E)
    bank = _bank(gen, E, H, I, shared)
    x = normal(gen, (T, H), torch.bfloat16)
    ids = torch.full((T, K), 2, dtype=torch.int32)
    ids[0], ids[1, 1], ids[T - 1, K - 1] = -1, E + 3, 0
    ids[2, :2] = torch.tensor([1, E - 1])
    assert (ids == 2).sum() > 16
    S = T * K + (T if shared else 0)
    y, (offsets, *_) = _check_experts(moe, bank, x, ids, E, H, I, shared,
                                      y_slots=torch.full((S, H), 5.0, dtype=torch.bfloat16, device="cuda"))
    end = int(offsets[-1])
    assert end == S - K - 1 and torch.equal(y[end:], torch.full_like(y[end:], 5.0))
    # a longer group is the same rows one after the other: bitwise those of a call with one row a token
    W = moe.FP8Weights(*(gpu(b) for b in bank), E, H, I, shared)
    one = torch.full((T, 1), 2, dtype=torch.int32)
    _, off1, ss1, pos1, gr1 = moe.moe_permute(gpu(one), E, shared)
    y1 = moe.moe_fp8_expert_ffn(W, gpu(x), 1, off1, ss1, gr1)
    G = lambda n: min(T * n, E) + int(shared)  # noqa: E731
    if (G(K) <= 16) == (G(1) <= 16) and (G(K) <= 48) == (G(1) <= 48):  # the same shapes, hence the same sums
        _, _, _, pos, _ = moe.moe_permute(gpu(ids), E, shared)
        for t in range(3, T - 1):
            for k in range(K):
                assert torch.equal(y[pos[t * K + k]].view(torch.int16), y1[pos1[t]].view(torch.int16))
