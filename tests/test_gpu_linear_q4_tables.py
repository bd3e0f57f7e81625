"""Tables of the 4-bit products by expert that moe_permute does not write."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native

pytestmark = pytest.mark.gpu


def test_more_active_experts_than_pairs_are_flagged():
    """Two pairs, six experts listed: no block looks at the last four, which is not kept quiet."""
    T, k, E, N, K, group = 1, 2, 6, 32, 64, 64
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    W = native.q4_weights(codes, torch.full((E, N, 1), 0.01).half().cuda(), None, group)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    tok = torch.zeros(2, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 0, 0, 0, 0, 1, 2], dtype=torch.int32, device="cuda")    # experts 4 and 5
    slots = torch.arange(E, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for listed, want in (([2, 4, 5, 0, 0, 0, 0], 0), ([6, 0, 1, 2, 3, 4, 5], native.DEV_BAD_INDEX)):
        active = torch.tensor(listed, dtype=torch.int32, device="cuda")
        out = torch.full((T * k, N), 7.0, device="cuda")
        status.zero_()
        native.expert_linear_q4(W, slots, x, T, E, k, offsets, tok, active, out, dev_status=status)
        assert int(status) == want
        assert (out == 7).any() == (want != 0)
