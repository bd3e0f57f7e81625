"""Calls of the 4-bit and the unquantised products from several host threads:
the same kernel with little and with much shared memory at the same time."""
import threading

import pytest
import torch

from bit_expert_ffn_fp32_b200 import native

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CALLS = 20000        # of each of four threads: an unlucky order of two calls is rare


def q4_call(K):
    """One row group and one token: the same kernel for every K, x staged in 2 to 64 steps."""
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 256, (1, 64, K // 2), generator=g, dtype=torch.uint8).cuda()
    scale = torch.full((1, 64, K // 64), 2.0 ** -6).half().cuda()
    W = native.q4_weights(codes, scale, None, 64)
    x = torch.randn(1, K, generator=g).to(BF).cuda()
    out = torch.empty(1, 64, dtype=F32, device="cuda")
    return lambda stream=None: native.linear_q4(W, 0, x, 1, out, stream=stream), out


def tables(E, rows):
    offsets = torch.full((E + 1,), rows, dtype=torch.int32)
    offsets[0] = 0
    return offsets.cuda()


def forward_call(E):
    """The table of experts lies in shared memory."""
    g = torch.Generator().manual_seed(E)
    W = torch.randn(E, 64, 64, generator=g).to(BF).cuda()
    a = torch.randn(8, 64, generator=g).to(BF).cuda()
    offsets, out = tables(E, 8), torch.empty(8, 64, dtype=F32, device="cuda")
    return lambda stream=None: native.expert_gemm(a, W, 8, E, 1, 64, 64, offsets, None, out, stream=stream), out


def wgrad_call(separate):
    """A sum so far that is read takes boxes of its own."""
    g = torch.Generator().manual_seed(5)
    E = 3
    dy, a = (torch.randn(100, 64, generator=g).to(BF).cuda() for _ in range(2))
    offsets, out = tables(E, 100), torch.empty(E, 64, 64, device="cuda")
    base = torch.randn(E, 64, 64, generator=g).cuda() if separate else None
    return lambda stream=None: native.expert_gemm_wgrad(dy, a, 100, E, 1, 64, 64, offsets, None, out, base=base,
                                                        stream=stream), out


PAIRS = {"q4": (q4_call, 64, 16384), "forward": (forward_call, 1, 4096), "wgrad": (wgrad_call, False, True)}


@pytest.mark.parametrize("name", PAIRS)
def test_host_threads(name):
    make, small, large = PAIRS[name]
    jobs = [make(small), make(large), make(small), make(large)]
    for call, _ in jobs:
        call()
    want = [out.clone() for _, out in jobs]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(jobs))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            for _ in range(CALLS):
                call(stream)
        except Exception as e:  # noqa: BLE001 (reported below, by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _ in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(torch.equal(out, w) for (_, out), w in zip(jobs, want))


@pytest.mark.parametrize("name", PAIRS)
def test_two_sizes_in_one_graph(name):
    make, small, large = PAIRS[name]
    jobs = [make(large), make(small), make(large)]
    for call, _ in jobs:
        call()
    want = [out.clone() for _, out in jobs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call, _ in jobs:
            call()
    for _ in range(3):
        for _, out in jobs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for (_, out), w in zip(jobs, want))
