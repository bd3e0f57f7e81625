"""The 4-bit products' SwiGLU where sig(gate) is a subnormal, or vanishes, in fp32
and the up row brings the result back: fp32 results keep their digits."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native
from routed import assert_close, silu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gates", [[-88.0, -92.0, -95.0, -96.0, -98.0, -99.0, -100.0, -102.0],
                                   [-103.0, -104.0, -105.0, -108.0, -110.0, -112.0, -120.0, -128.0]])
def test_far_gates(gates):
    """Gate -8 s x_0 and up 2^15 2^112 are exact. exp of half the gate is off by two
    steps of 2^-23 at most and enters twice; three products, one sum and a
    division round once each: below 2^-20."""
    gate = torch.tensor(gates).repeat(4)
    codes = torch.full((64, 128), 0x88, dtype=torch.uint8)      # every weight zero but
    codes[:32, 0], codes[32:, 64] = 0x80, 0x89                  # weight 0 of the gates, -8, and 128 of the up rows, 1
    scale = torch.zeros(64, 2)
    scale[:32, 0], scale[32:, 1] = gate / -8, 2.0 ** 15
    assert torch.equal(scale.half().float(), scale)
    x = torch.zeros(1, 256, dtype=torch.bfloat16)
    x[0, 0], x[0, 128] = 1.0, 2.0 ** 112
    out = torch.empty(1, 32, device="cuda")
    native.linear_q4(native.q4_weights(codes.cuda(), scale.half().cuda(), None, 128), 0, x.cuda(), 1, out,
                     native.ACT_SWIGLU)
    want = (silu(gate.double()) * 2.0 ** 127)[None].cuda()
    assert (want.abs() > 2.0 ** -60).all()
    assert_close(out, want, want.abs() * 2.0 ** -20)
