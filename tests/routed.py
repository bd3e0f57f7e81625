"""Routed batches and 64-bit references shared by the tests of the 4-bit and
the unquantised expert products."""
from __future__ import annotations

import torch

EPS2 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half the least step


def route(T, k, E, seed, crowd=0.0, device="cuda"):
    """idx [T][k] (ascending, distinct), offsets, sorted_tok, active, as moe_permute
    leaves them; a share `crowd` of the tokens choose expert 0."""
    g = torch.Generator().manual_seed(seed)
    score = torch.rand(T, E, generator=g)
    score[: int(crowd * T), 0] = 2.0
    idx = torch.sort(torch.topk(score, k, dim=1).indices, dim=1).values if T else torch.zeros(0, k, dtype=torch.long)
    order = torch.sort(idx.reshape(-1), stable=True)
    counts = torch.bincount(order.values, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    offsets[1:] = torch.cumsum(counts, 0)
    ids = torch.nonzero(counts).reshape(-1)
    active = torch.full((E + 1,), -7, dtype=torch.int32)   # past the list: never read
    active[0] = ids.numel()
    active[1: 1 + ids.numel()] = ids
    tok = (order.indices // k).to(torch.int32)
    return idx, offsets.to(device), tok.to(device), active.to(device)


def ranges(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def sum_bound(inner):
    """Error of a sum of `inner` products relative to the sum of their magnitudes:
    at most inner / 16 + 32 additions follow one another, each off by no more
    than a whole step of fp32 (tensor cores may cut instead of round)."""
    return (inner / 16 + 32) * 2.0 ** -23


def assert_close(got, want, tol):
    """|got - want| <= tol + the rounding of got's type, element by element."""
    got64 = got.double()
    tol = tol + EPS2[got.dtype] * want.abs() * (1 + 1e-6) + TINY[got.dtype]
    bad = ~((got64 - want).abs() <= tol)
    assert not bad.any(), (
        f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: "
        f"{got64[bad][0].item()} for {want[bad][0].item()}, allowed {tol[bad][0].item()}")


def silu(x):
    return x * torch.special.expit(x)
