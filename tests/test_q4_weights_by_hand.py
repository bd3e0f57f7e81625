"""A description of 4-bit weights whose addresses the caller filled in."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native

BF = torch.bfloat16


def test_host_tensors_are_refused():
    W = native.Q4Weights(0x10000, 0x10000, None, 2, 64, 128, 64)
    x, out, table = torch.zeros(1, 128, dtype=BF), torch.zeros(1, 64, dtype=BF), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        native.linear_q4(W, 0, x, 1, out)
    with pytest.raises(ValueError):
        native.expert_linear_q4(W, table, x, 1, 2, 1, table, None, table, out)


@pytest.mark.gpu
def test_same_results():
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 256, (2, 64, 64), generator=g, dtype=torch.uint8).cuda()
    scale = torch.rand(2, 64, 2, generator=g).half().cuda()
    x = torch.randn(2, 128, generator=g).to(BF).cuda()
    by_hand = native.Q4Weights(codes.data_ptr(), scale.data_ptr(), None, 2, 64, 128, 64)
    offsets = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    active, slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda"), torch.arange(2, device="cuda").int()
    got = []
    for W in (native.q4_weights(codes, scale, None, 64), by_hand):
        y, z = torch.empty(2, 64, dtype=BF, device="cuda"), torch.empty(2, 64, dtype=BF, device="cuda")
        native.linear_q4(W, 1, x, 2, y)
        native.expert_linear_q4(W, slots, x, 2, 2, 1, offsets, None, active, z)
        got.append((y, z))
    assert all(torch.equal(a, b) for a, b in zip(*got))
