"""Refusals of the 4-bit and the unquantised products and of SwiGLU, before
anything is enqueued: no GPU is needed, and no address is read."""
import ctypes as C

import pytest
import torch

from bit_expert_ffn_fp32_b200 import native

L = native.lib
A = 0x10000            # an aligned address that is never read
INVALID, UNSUPPORTED, OVERFLOW = 1, 2, 5


def q4(**kw):
    w = dict(codes=A, scale=A, min=A, num_slots=4, N=64, K=128, group=64)
    w.update(kw)
    return native.Q4Weights(*w.values())


def dense(w=None, slot=0, x=A, dtype=0, T=2, act=0, out=A, out_dtype=0):
    return L.moe_linear_q4(C.addressof(w) if w is not None else None, slot, x, dtype, T, act, out, out_dtype, None)


def by_expert(w, slot_of=A, x=A, dtype=0, T=2, E=8, k=2, offsets=A, tok=A, active=A, act=0, out=A, out_dtype=0):
    return L.moe_expert_linear_q4(C.addressof(w), slot_of, x, dtype, T, E, k, offsets, tok, active, act, out, out_dtype,
                                  None, None)


def test_q4_refusals():
    assert dense(None) == INVALID
    for kw in (dict(codes=None), dict(scale=None), dict(codes=A + 8), dict(scale=A + 1), dict(min=A + 1),
               dict(num_slots=0), dict(N=0), dict(K=-64)):
        assert dense(q4(**kw)) == INVALID, kw
    for kw in (dict(group=16), dict(group=256, K=256), dict(N=48), dict(K=96), dict(N=16416), dict(K=16512)):
        assert dense(q4(**kw)) == UNSUPPORTED, kw
    ok = q4()
    for kw in (dict(slot=4), dict(slot=-1), dict(x=None), dict(x=A + 2), dict(out=None), dict(out=A + 8), dict(T=-1),
               dict(dtype=2), dict(dtype=3), dict(out_dtype=1), dict(act=2)):
        assert dense(ok, **kw) == INVALID, kw
    assert dense(ok, T=0, x=None, out=None) == 0
    for kw in (dict(slot_of=None), dict(offsets=None), dict(active=None), dict(x=None), dict(out=None), dict(x=A + 4),
               dict(E=0), dict(k=0), dict(T=-1)):
        assert by_expert(ok, **kw) == INVALID, kw
    for kw in (dict(E=4097), dict(k=17, E=32), dict(k=9)):
        assert by_expert(ok, **kw) == UNSUPPORTED, kw
    assert by_expert(ok, T=1 << 30) == OVERFLOW and by_expert(ok, T=(1 << 31) - 4095, k=1) == OVERFLOW
    assert dense(ok, T=(1 << 31) - 1) == OVERFLOW
    assert by_expert(ok, T=0, x=None, out=None) == 0


GEMM = dict(x=A, y=A, dtype=0, T=2, E=8, k=2, N=64, K=64, offsets=A, out=A, out_dtype=0)


def forward(**kw):
    c = {**GEMM, **kw}
    return L.moe_expert_gemm(c["x"], c["y"], c["dtype"], c["T"], c["E"], c["k"], c["N"], c["K"], c["offsets"], None,
                             c["out"], c["out_dtype"], None, None)


def dgrad(**kw):
    c = {**GEMM, **kw}
    return L.moe_expert_gemm_dgrad(c["x"], c["y"], c["dtype"], c["T"], c["E"], c["k"], c["N"], c["K"], c["offsets"],
                                   c["out"], c["out_dtype"], None, None)


def wgrad(base=None, **kw):
    c = {**GEMM, **kw}
    return L.moe_expert_gemm_wgrad(c["x"], c["y"], c["dtype"], c["T"], c["E"], c["k"], c["N"], c["K"], c["offsets"],
                                   None, base, c["out"], c["out_dtype"], None, None)


@pytest.mark.parametrize("call", [forward, dgrad, wgrad])
def test_gemm_refusals(call):
    for kw in (dict(x=None), dict(y=None), dict(offsets=None), dict(out=None), dict(x=A + 2), dict(y=A + 8),
               dict(out=A + 4), dict(T=-1), dict(E=0), dict(k=0), dict(N=0), dict(K=-8), dict(dtype=2),
               dict(out_dtype=1), dict(dtype=1, out_dtype=0), dict(dtype=-1, out_dtype=-1)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(N=60), dict(K=68), dict(N=16392), dict(K=16392), dict(E=4097), dict(k=17, E=32), dict(k=9)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(T=1 << 30) == OVERFLOW and call(T=(1 << 31) - 4095, k=1) == OVERFLOW


def test_gemm_of_no_tokens():
    assert forward(T=0, x=None, y=None, out=None) == 0
    assert dgrad(T=0, x=None, y=None, out=None) == 0
    assert wgrad(T=0, out=None) == INVALID        # dW is written for every expert
    assert wgrad(base=A + 4) == INVALID


def test_swiglu_refusals():
    f, b = L.moe_swiglu, L.moe_swiglu_backward
    for args in ((None, 0, 4, 64, A), (A, 0, 4, 64, None), (A + 2, 0, 4, 64, A), (A, 0, 4, 64, A + 8),
                 (A, 2, 4, 64, A), (A, 0, -1, 64, A), (A, 0, 4, 0, A)):
        assert f(*args, None) == INVALID, args
    assert f(A, 0, 4, 60, A, None) == UNSUPPORTED and f(A, 0, 4, 16392, A, None) == UNSUPPORTED
    assert f(A, 0, 1 << 31, 64, A, None) == OVERFLOW
    assert f(None, 0, 0, 64, None, None) == 0 and b(None, None, 0, 0, 64, None, None) == 0
    for args in ((None, A, 0, 4, 64, A), (A, None, 0, 4, 64, A), (A, A, 0, 4, 64, None), (A, A + 2, 0, 4, 64, A),
                 (A, A, 0, 4, 64, A + 2), (A, A, 2, 4, 64, A)):
        assert b(*args, None) == INVALID, args


def test_binding_refusals():
    """The binding looks at types, sizes and places before an address leaves it."""
    z = torch.zeros
    bf = torch.bfloat16
    for bad in (dict(codes=z(2, 64, 64)), dict(scale=z(2, 64, 3).half()), dict(min=z(2, 64, 2)), dict(group=48),
                dict(group=256), dict(codes=z(2, 64, 128, dtype=torch.uint8)[:, :, ::2])):
        kw = dict(codes=z(2, 64, 64, dtype=torch.uint8), scale=z(2, 64, 2).half(), min=None, group=64)
        kw.update(bad)
        with pytest.raises(ValueError):
            native.q4_weights(**kw)
    W = native.q4_weights(z(2, 64, 64, dtype=torch.uint8), z(2, 64, 2).half(), None, 64)
    assert (W.N, W.K, W.num_slots, W.group) == (64, 128, 2, 64)
    with pytest.raises(ValueError):                # host tensors
        native.linear_q4(W, 0, z(1, 128, dtype=bf), 1, z(1, 64, dtype=bf))
    with pytest.raises(ValueError):
        native.swiglu(z(4, 128, dtype=bf), 4, 64, z(4, 64, dtype=bf))
    with pytest.raises(ValueError):
        native.dtype_code(z(2, dtype=torch.float64))
