"""fp32 results of the 4-bit products against the sums they are formed from: s*q
and m of a group with min, s*(q-8) without."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native
from routed import assert_close

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def make(N, K, group, with_min, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (1, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scale = ((0.5 + torch.rand(1, N, K // group, generator=g)) / (4.6 * K ** 0.5)).half().cuda()
    mn = None
    if with_min:
        mn = (-7.5 * scale.float() * (0.8 + 0.4 * torch.rand(1, N, K // group, generator=g).cuda())).half()
    return codes, scale, mn


def weights(codes, scale, mn, group):
    """W, and the magnitude of what each weight is the sum of."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double()[0]
    s = scale.double().repeat_interleave(group, dim=-1)[0]
    if mn is None:
        return s * (q - 8), (s * (q - 8)).abs()
    m = mn.double().repeat_interleave(group, dim=-1)[0]
    return s * q + m, s * q + m.abs()


def run(parts, group, x, N):
    out = torch.empty(x.shape[0], N, device="cuda")
    native.linear_q4(native.q4_weights(*parts, group), 0, x, x.shape[0], out)
    return out


def bound(K, group):
    """Additions one behind another, each off by a whole step of fp32 at most (tensor
    cores may cut): those inside a group, those of the groups, and scale, offset
    and the joining of the warps' sums."""
    return (K / 16 + K / group + 40) * 2.0 ** -23


@pytest.mark.parametrize("with_min", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K,T,dtype", [(64, 384, 1, BF), (512, 2048, 3, FP), (2048, 768, 9, BF), (96, 16384, 20, FP),
                                         (1536, 2048, 40, BF)])
def test_against_its_terms(with_min, group, N, K, T, dtype):
    """Element by element against the terms' magnitudes; and by norms: a group's sum
    takes at most 8 products of 16, each cutting half a step of the sum so far on
    average, which grows with the root of the count: (1/2)(2/3) 8 steps; the rest
    rounds to nearest, three steps at most: 6 steps of the terms' norm."""
    parts = make(N, K, group, with_min, N + group)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(K)).to(dtype).cuda()
    out = run(parts, group, x, N)
    W, mag = weights(*parts, group)
    want = x.double() @ W.t()
    assert_close(out, want, (x.double().abs() @ mag.t()) * bound(K, group))
    terms = (x.double() ** 2 @ (mag ** 2).t()).sum().sqrt()
    assert (out.double() - want).norm() <= 6 * 2.0 ** -23 * terms


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("outlier", [2.0 ** 12, -2.0 ** 14])
def test_outlier_on_zero_weights(group, dtype, outlier):
    """Without min a weight of zero is a product of zero, whatever x: the others keep
    the digits that they have without it, but for their rounding: scaled so that the
    largest is 2^10 or more, to half of fp16's smallest step, 2^-25."""
    N, K = 64, 512
    codes, scale, _ = make(N, K, group, False, 8)
    codes[0, :, 50] = 0x88                               # weights 100 and 101 are 0
    x = (torch.randn(3, K, generator=torch.Generator().manual_seed(1)) * 2.0 ** -8).to(dtype).cuda()
    x[:, 100], x[:, 101] = outlier, -outlier / 2
    out = run((codes, scale, None), group, x, N)
    W, mag = weights(codes, scale, None, group)
    x0 = x.double()
    x0[:, 100:102] = 0
    want = x0 @ W.t()
    assert_close(out, want, (x0.abs() @ mag.t()) * bound(K, group) + 2.0 ** -35 * abs(outlier) * mag.sum(dim=1))


@pytest.mark.parametrize("T", [1, 3, 12, 40])
def test_every_code(T):
    """All sixteen codes in both halves of a byte, on powers of two: exact."""
    K, group, N = 512, 64, 32
    codes = torch.arange(256, dtype=torch.uint8).repeat(N, 1)
    for i in range(N):
        codes[i] = codes[i].roll(7 * i)
    scale = torch.full((N, K // group), 0.5).half()
    x = torch.randint(-3, 4, (T, K), generator=torch.Generator().manual_seed(T)).to(BF).cuda()
    for mn in (None, torch.full((N, K // group), -3.25).half().cuda()):
        parts = (codes[None].cuda(), scale[None].cuda(), None if mn is None else mn[None])
        out = run(parts, group, x, N)
        assert torch.equal(out.double(), x.double() @ weights(*parts, group)[0].t())
