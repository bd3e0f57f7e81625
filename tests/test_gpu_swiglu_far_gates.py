"""SwiGLU where sig(gate) is a subnormal and the up value brings the result back."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native
from routed import assert_close

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
GATES = [-95.0, -98.0, -98.5, -99.0, -100.0, -101.5, -102.0, -103.0]


@pytest.mark.parametrize("up", [2.0 ** 124, -2.0 ** 127])
def test_far_gates(up):
    """Forward: exp's argument, up to 149 in powers of two, is off by 2^-17 and its
    constant's 149 * 2^-26, times ln 2; sig keeps 15 bits; exp2, division and two
    products add 2^-21: below 2^-14.5 together. Backward: the same, and sig's
    subnormals are off by half a step twice (exp, the product with 1 / (1 + exp))."""
    g = torch.tensor([GATES], device="cuda").to(BF)
    assert g.double().flatten().tolist() == GATES
    u, dh = torch.full_like(g, up), torch.full_like(g, 0.5)
    gu = torch.cat((g, u), dim=1)
    h, dgu = torch.empty(1, 8, dtype=BF, device="cuda"), torch.empty(1, 16, dtype=BF, device="cuda")
    native.swiglu(gu, 1, 8, h)
    native.swiglu_backward(gu, dh, 1, 8, dgu)
    g, u, dh = g.double(), u.double(), dh.double()
    s = torch.special.expit(g)
    want = g * s * u
    assert (want.abs() > 2.0 ** -18).all()
    assert_close(h, want, want.abs() * 2.0 ** -14.5)
    slope = torch.cat((dh * u * (1 + g * (1 - s)), dh * g), dim=1)
    want = slope * s.repeat(1, 2)
    assert_close(dgu, want, want.abs() * 2.0 ** -14.5 + slope.abs() * 2.0 ** -149)


def test_scaled_up_values_are_exact():
    """The forward scales u on its way: subnormal, tiny and huge u lose nothing."""
    u = torch.tensor([2.0 ** -133, 3 * 2.0 ** -132, 1.9921875 * 2.0 ** -126, 2.0 ** -100, 2.0 ** -30, 1.0,
                      1.9921875 * 2.0 ** 127, -1.9921875 * 2.0 ** 127], dtype=torch.float64)
    for gate in (1.0, 64.0, -0.5, -4.0):
        g = torch.full((1, 8), gate, device="cuda").to(BF)
        gu = torch.cat((g, u[None].cuda().to(BF)), dim=1)
        assert torch.equal(gu[0, 8:].double().cpu(), u)
        h = torch.empty(1, 8, dtype=BF, device="cuda")
        native.swiglu(gu, 1, 8, h)
        want = torch.special.expit(g.double()) * g.double() * u.cuda()
        fits = want.abs() < 2.0 ** 128
        assert_close(h[fits], want[fits], want[fits].abs() * 2.0 ** -18 + 2.0 ** -150 * abs(gate))
        assert torch.isinf(h[~fits]).all()
