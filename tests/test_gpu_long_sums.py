"""Long sums of the unquantised products, by norms: the error must not grow with
the length of the contracted index or with the rows of a crowded expert.

The tensor cores add 16 products at a time and cut. A cut takes half a step of
the sum so far on average, a step is at most 2^-23 of it, and a sum of random
terms grows with the root of their count: n additions lose (1/2) (2/3) n steps
of the last sum. fp32 results come from chains of 64 additions at most, 21.4
steps; joining the chains rounds to nearest, below 2.6 steps: 24 * 2^-23. 16-bit
results come from chains of 1024 additions, and are rounded once."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
FP32_TOL = 24 * 2.0 ** -23


def rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def table(rows):
    offsets = torch.zeros(len(rows) + 1, dtype=torch.int32)
    offsets[1:] = torch.cumsum(torch.tensor(rows), 0)
    return offsets.cuda()


def error(got, want):
    return float((got.double() - want).norm() / want.norm())


# experts x rows each: narrow tiles, wide ones (one of several tiles), a mixture that is wide
@pytest.mark.parametrize("rows", [[5, 16], [300, 129], [1, 600, 40]])
@pytest.mark.parametrize("inner", [768, 1032, 2048, 4104, 16384])
@pytest.mark.parametrize("dtype,gather", [(BF, True), (FP, False)])
def test_long_contractions(rows, inner, dtype, gather):
    E, P, outer = len(rows), sum(rows), 136
    offsets, tok = table(rows), torch.arange(P, dtype=torch.int32, device="cuda").flip(0).contiguous()
    x = rand((P, inner), dtype, 1)
    W, Wt = rand((E, outer, inner), dtype, 2), rand((E, inner, outer), dtype, 3)
    out, da = torch.empty(P, outer, device="cuda"), torch.empty(P, outer, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.expert_gemm(x, W, P, E, 1, outer, inner, offsets, tok if gather else None, out, dev_status=status)
    native.expert_gemm_dgrad(x, Wt, P, E, 1, inner, outer, offsets, da, dev_status=status)
    a, r0 = (x[tok.long()] if gather else x).double(), 0
    want, dwant = torch.empty_like(out, dtype=torch.float64), torch.empty_like(out, dtype=torch.float64)
    for e, n in enumerate(rows):
        want[r0:r0 + n] = a[r0:r0 + n] @ W[e].double().t()
        dwant[r0:r0 + n] = x[r0:r0 + n].double() @ Wt[e].double()
        r0 += n
    assert int(status) == 0
    assert error(out, want) <= FP32_TOL and error(da, dwant) <= FP32_TOL


@pytest.mark.parametrize("rows", [[4133] + [9] * 63, [7, 0, 20000, 300, 1024, 1025, 0], [65, 2048, 2049]])
@pytest.mark.parametrize("gather,base", [(True, None), (False, "in place"), (True, "separate")])
def test_crowded_expert(rows, gather, base):
    """The weight gradient of an expert with many rows, whatever the others have."""
    E, P, N, K = len(rows), sum(rows), 72, 264
    offsets, tok = table(rows), torch.arange(P, dtype=torch.int32, device="cuda").flip(0).contiguous()
    dy, a = rand((P, N), BF, 1), rand((P, K), BF, 2)
    before = rand((E, N, K), F32, 3) if base else None
    dW = before.clone() if base == "in place" else torch.empty(E, N, K, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.expert_gemm_wgrad(dy, a, P, E, 1, N, K, offsets, tok if gather else None, dW,
                             base=dW if base == "in place" else before, dev_status=status)
    x, r0 = (a[tok.long()] if gather else a).double(), 0
    for e, n in enumerate(rows):
        want = dy[r0:r0 + n].double().t() @ x[r0:r0 + n]
        want = want + before[e].double() if base else want
        assert error(dW[e], want) <= FP32_TOL if n else torch.equal(dW[e].double(), want), (e, n)
        r0 += n
    assert int(status) == 0


@pytest.mark.parametrize("separate", [False, True])
def test_16_bit_results_of_very_many_rows(separate):
    """600,000 rows: cutting alone would pass half a step of fp16. Of 1024 additions it
    is (1/2) (2/3) 1024 * 2^-23 = 4.1e-5; rounding, evenly spread over half a step,
    at most 2^-11 / sqrt(3) = 2.82e-4: 2.85e-4 together, 3e-4 with its spread over
    12,288 values."""
    rows = [600000, 17000, 40]
    E, P, N, K = len(rows), sum(rows), 64, 64
    offsets, dy, a = table(rows), rand((P, N), FP, 1), rand((P, K), FP, 2)
    base = rand((E, N, K), FP, 3) if separate else None
    dW = torch.empty(E, N, K, dtype=FP, device="cuda")
    native.expert_gemm_wgrad(dy, a, P, E, 1, N, K, offsets, None, dW, base=base)
    r0 = 0
    for e, n in enumerate(rows):
        want = dy[r0:r0 + n].double().t() @ a[r0:r0 + n].double()
        want = want + base[e].double() if separate else want
        assert error(dW[e], want) <= 3e-4, (e, n)
        r0 += n


def test_equal_bits_and_graphs():
    """Tiles of one and of several segments in turn, in a replayed graph."""
    rows = [40, 3000, 0, 1500, 17, 1024]
    E, P, N, K = len(rows), sum(rows), 320, 200
    offsets, dy, a = table(rows), rand((P, N), BF, 1), rand((P, K), BF, 2)
    W = rand((E, N, 4096), BF, 3)
    x, out = rand((P, 4096), BF, 4), torch.empty(P, N, device="cuda")
    dW = torch.empty(E, N, K, device="cuda")

    def both():
        native.expert_gemm_wgrad(dy, a, P, E, 1, N, K, offsets, None, dW)
        native.expert_gemm(x, W, P, E, 1, N, 4096, offsets, None, out)

    both()
    want = dW.clone(), out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        dW.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dW, want[0]) and torch.equal(out, want[1])
