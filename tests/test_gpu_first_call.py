"""The first call that a host thread makes: nothing before it has made the
device's context current there."""
import threading

import pytest
import torch

from bit_expert_ffn_fp32_b200 import configs, native, synth
from bit_expert_ffn_fp32_b200.layer import MoEStack, x_tensor

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def products():
    """name -> (call(stream), its output)."""
    E, P, N, K = 3, 60, 64, 64
    g = torch.Generator().manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=g).to(BF).cuda()

    offsets = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device="cuda")
    a, W, dy = rand(P, K), rand(E, N, K), rand(P, N)
    out, da, dW = (torch.empty(*s, device="cuda") for s in ((P, N), (P, K), (E, N, K)))
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8).cuda()
    W4 = native.q4_weights(codes, torch.full((N, K // 64), 0.01).half().cuda(), None, 64)
    y4 = torch.empty(P, N, device="cuda")
    gu, h = rand(P, 2 * 64), torch.empty(P, 64, dtype=BF, device="cuda")
    return {
        "expert_gemm": (lambda s: native.expert_gemm(a, W, P, E, 1, N, K, offsets, None, out, stream=s), out),
        "expert_gemm_dgrad": (lambda s: native.expert_gemm_dgrad(dy, W, P, E, 1, N, K, offsets, da, stream=s), da),
        "expert_gemm_wgrad": (lambda s: native.expert_gemm_wgrad(dy, a, P, E, 1, N, K, offsets, None, dW, stream=s),
                              dW),
        "linear_q4": (lambda s: native.linear_q4(W4, 0, a, P, y4, stream=s), y4),
        "swiglu": (lambda s: native.swiglu(gu, P, 64, h, stream=s), h),
    }


def decode():
    stack = MoEStack(configs.TINY)
    x, b = x_tensor(synth.gen_x(1, 0, 4, stack.wl.d), stack.device), stack.buffers(4)
    return {"layer_decode": (lambda s: stack.forward_fused(0, x, b, stream=s), b.y)}


@pytest.mark.parametrize("make,name", [(products, n) for n in ("expert_gemm", "expert_gemm_dgrad", "expert_gemm_wgrad",
                                                               "linear_q4", "swiglu")] + [(decode, "layer_decode")])
def test_first_call_of_a_host_thread(make, name):
    call, out = make()[name]
    stream = torch.cuda.Stream()
    call(stream)                       # the kernel and the encoder are known
    stream.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call(stream)
        except Exception as e:  # noqa: BLE001 (reported below, by the test's own thread)
            errors.append(e)

    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert not errors, errors
    if name == "layer_decode":         # its partial sums meet in any order
        assert (out - want).abs().max() <= 1e-5 * want.abs().max()
    else:
        assert torch.equal(out, want)
