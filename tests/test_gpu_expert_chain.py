"""The operators as they are used together: a routed layer through moe_route and
moe_permute, its experts in 16 bits forward and backward, its experts in 4 bits,
and moe_combine, against the layer's formula in 64 bits."""
import numpy as np
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native, synth
from routed import silu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def routed(T, d, E, k):
    """x (bf16) and its routing by the library, on the GPU."""
    x = torch.from_numpy(synth.gen_x(3, 0, T, d, stream=1).view(np.int16)).cuda().view(BF)
    Wr = torch.from_numpy(synth.gen_router(3, 0, E, d)).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    logits = torch.empty(T, E, device="cuda")
    idx, w = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    counts, offsets, active = (torch.empty(E + 1, **i32) for _ in range(3))
    tok, j, inv = (torch.empty(T * k, **i32) for _ in range(3))
    need = native.permute_workspace_bytes(T, k, E)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    native.route(x, Wr, None, T, d, E, k, logits, idx, w)
    native.permute(idx, T, k, E, counts, offsets, tok, j, inv, active, ws, need)
    return x, idx, w, offsets, tok, inv, active


def close(got, want, tol):
    err = float((got.double() - want).norm() / want.norm())
    assert err <= tol, err


@pytest.mark.parametrize("T", [1, 5, 16, 200])
def test_layer_in_16_bits_and_its_gradients(T):
    """h and every gradient between the products is rounded to bf16 once (2^-8 of
    each value at most); four such roundings meet in the last gradient."""
    d, f, E, k = 256, 256, 32, 4
    P = T * k
    x, idx, w, offsets, tok, inv, _ = routed(T, d, E, k)
    g = torch.Generator().manual_seed(1)
    Wgu = (torch.randn(E, 2 * f, d, generator=g) / d ** 0.5).to(BF).cuda()
    Wd = (torch.randn(E, d, f, generator=g) / f ** 0.5).to(BF).cuda()
    dy = torch.randn(T, d, generator=g).cuda()
    gu, h = torch.empty(P, 2 * f, dtype=BF, device="cuda"), torch.empty(P, f, dtype=BF, device="cuda")
    y_perm, y = torch.empty(P, d, device="cuda"), torch.empty(T, d, device="cuda")
    native.expert_gemm(x, Wgu, T, E, k, 2 * f, d, offsets, tok, gu)
    native.swiglu(gu, P, f, h)
    native.expert_gemm(h, Wd, T, E, k, d, f, offsets, None, y_perm)
    native.combine(y_perm, inv, w, None, None, T, k, d, y)

    # backward: the gradient of pair s is its gate times the token's
    pair_of = torch.empty(P, dtype=torch.long, device="cuda")
    pair_of[inv.long()] = torch.arange(P, device="cuda")
    dyp = (w.reshape(-1)[pair_of, None] * dy[pair_of // k]).to(BF)
    dh, dgu = torch.empty(P, f, dtype=BF, device="cuda"), torch.empty(P, 2 * f, dtype=BF, device="cuda")
    dWd, dWgu = torch.empty(E, d, f, device="cuda"), torch.empty(E, 2 * f, d, device="cuda")
    dxp, dx = torch.empty(P, d, device="cuda"), torch.empty(T, d, device="cuda")
    native.expert_gemm_dgrad(dyp, Wd, T, E, k, d, f, offsets, dh)
    native.expert_gemm_wgrad(dyp, h, T, E, k, d, f, offsets, None, dWd)
    native.swiglu_backward(gu, dh, P, f, dgu)
    native.expert_gemm_dgrad(dgu, Wgu, T, E, k, 2 * f, d, offsets, dxp)
    native.expert_gemm_wgrad(dgu, x, T, E, k, 2 * f, d, offsets, tok, dWgu)
    native.combine(dxp, inv, torch.ones_like(w), None, None, T, k, d, dx)

    X, G, D = x.double().requires_grad_(), Wgu.double().requires_grad_(), Wd.double().requires_grad_()
    want = 0
    for j in range(k):
        e = idx[:, j].long()
        gu64 = torch.einsum("tnd,td->tn", G[e], X)
        want = want + w[:, j, None].double() * torch.einsum("tdf,tf->td", D[e], silu(gu64[:, :f]) * gu64[:, f:])
    want.backward(dy.double())
    close(y, want.detach(), 3 * 2.0 ** -8)
    for got, ref in ((dx, X.grad), (dWd, D.grad), (dWgu, G.grad)):
        close(got, ref, 4 * 2.0 ** -8)


@pytest.mark.parametrize("T", [1, 4, 37])
def test_layer_in_4_bits(T):
    """h is the only value between the products that is rounded to bf16."""
    d, f, E, k, group = 512, 256, 64, 4, 64
    P = T * k
    x, idx, w, offsets, tok, inv, active = routed(T, d, E, k)
    g = torch.Generator().manual_seed(2)

    def pool(N, K):
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8).cuda()
        scale = (torch.rand(E, N, K // group, generator=g) / (4.6 * K ** 0.5)).half().cuda()
        q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double()
        return native.q4_weights(codes, scale, None, group), (q - 8) * scale.double().repeat_interleave(group, -1)

    (gu_w, GU), (d_w, D) = pool(2 * f, d), pool(d, f)
    slot_of = torch.arange(E, dtype=torch.int32, device="cuda")
    h, y_perm = torch.empty(P, f, dtype=BF, device="cuda"), torch.empty(P, d, device="cuda")
    y = torch.empty(T, d, device="cuda")
    native.expert_linear_q4(gu_w, slot_of, x, T, E, k, offsets, tok, active, h, native.ACT_SWIGLU)
    native.expert_linear_q4(d_w, slot_of, h, T, E, k, offsets, None, active, y_perm)
    native.combine(y_perm, inv, w, None, None, T, k, d, y)
    want = 0
    for j in range(k):
        e = idx[:, j].long()
        gu = torch.einsum("tnd,td->tn", GU[e], x.double())
        want = want + w[:, j, None].double() * torch.einsum("tdf,tf->td", D[e], silu(gu[:, :f]) * gu[:, f:])
    close(y, want, 2.0 ** -8)
