"""Products with 4-bit weights, dense and grouped by expert, against the
definition in 64 bits."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native
from routed import assert_close, ranges, route, silu

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def make(slots, N, K, group, with_min, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (slots, N, K // 2), generator=g, dtype=torch.uint8).cuda()
    scale = ((0.5 + torch.rand(slots, N, K // group, generator=g)) / (4.6 * K ** 0.5)).half().cuda()
    mn = None
    if with_min:
        mn = (-7.5 * scale.float() * (0.8 + 0.4 * torch.rand(slots, N, K // group, generator=g).cuda())).half()
    return codes, scale, mn


def dense(codes, scale, mn, group):
    """W and, for the error bound, the magnitude the products may be formed from:
    codes shifted by 16 and the shift taken off again, (16 + q) s and |m - 16 s|."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double()
    s = scale.double().repeat_interleave(group, dim=-1)
    m = mn.double().repeat_interleave(group, dim=-1) if mn is not None else -8 * s
    return s * q + m, s.abs() * (16 + q) + (m - 16 * s).abs()


def bound(K, group):
    """As for a plain sum (tests/routed.py), by group: the additions inside a group,
    those of the groups, and two more for scale and offset."""
    return (K / 16 + K / group + 40) * 2.0 ** -23


def reference(parts, group, act, slot, x):
    codes, scale, mn = parts
    W, mag = dense(codes[slot], scale[slot], None if mn is None else mn[slot], group)
    x = x.double()
    y, tol = x @ W.t(), (x.abs() @ mag.t()) * bound(x.shape[1], group)
    if act == native.ACT_NONE:
        return y, tol
    g, u = y.chunk(2, dim=1)
    tg, tu = tol.chunk(2, dim=1)
    h = silu(g) * u                                     # |silu'| <= 1.1
    return h, 1.1 * tg * (u.abs() + tu) + silu(g).abs() * tu + h.abs() * 2.0 ** -18


SIZES = [(32, 32, 32), (64, 64, 64), (96, 1056, 32), (160, 704, 64), (256, 640, 128), (1536, 2048, 64),
         (2048, 768, 128), (64, 8192, 64), (32, 16384, 128), (1088, 256, 32)]


@pytest.mark.parametrize("N,K,group", SIZES)
@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 17, 40, 130])
@pytest.mark.parametrize("with_min,act,dtype,out_dtype", [(True, 0, BF, BF), (False, 1, BF, F32), (True, 1, FP, FP),
                                                          (False, 0, FP, F32)])
def test_dense(N, K, group, T, with_min, act, dtype, out_dtype):
    parts = make(3, N, K, group, with_min, seed=N + K)
    x = rand((T, K), dtype, T)
    out = torch.full((T + 1, N // (1 + act)), 7.0, dtype=out_dtype, device="cuda")
    native.linear_q4(native.q4_weights(*parts, group), 1, x, T, out, act)
    assert_close(out[:T], *reference(parts, group, act, 1, x))
    assert (out[T] == 7).all()


@pytest.mark.parametrize("T,k,E,crowd", [(1, 1, 1, 0.0), (1, 10, 64, 0.0), (4, 10, 40, 1.0), (37, 3, 9, 0.6),
                                         (64, 16, 100, 0.2), (300, 2, 8, 0.7)])
@pytest.mark.parametrize("N,K,group,with_min,act", [(256, 512, 64, True, 1), (160, 288, 32, False, 0),
                                                    (512, 256, 128, True, 0)])
@pytest.mark.parametrize("gather,dtype,out_dtype", [(True, BF, BF), (False, FP, F32), (False, BF, F32)])
def test_by_expert(T, k, E, crowd, N, K, group, with_min, act, gather, dtype, out_dtype):
    _, offsets, tok, active = route(T, k, E, seed=T + E, crowd=crowd)
    P, S = T * k, E + 3
    parts = make(S, N, K, group, with_min, seed=E)
    slot_of = torch.randperm(S, generator=torch.Generator().manual_seed(E))[:E].to(torch.int32)
    slot_of[1::3] = -1                                   # a third of the experts has no slot
    x = rand((T if gather else P, K), dtype, 1)
    out = torch.full((P, N // (1 + act)), 7.0, dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.expert_linear_q4(native.q4_weights(*parts, group), slot_of.cuda(), x, T, E, k, offsets,
                            tok if gather else None, active, out, act, dev_status=status)
    assert int(status) == 0
    for e, r0, r1 in ranges(offsets):
        slot = int(slot_of[e])
        if slot < 0:
            assert (out[r0:r1] == 7).all()
        else:
            rows = x[tok[r0:r1].long()] if gather else x[r0:r1]
            assert_close(out[r0:r1], *reference(parts, group, act, slot, rows))


def test_bad_tables_are_flagged_and_skipped():
    T, k, E, N, K, group = 12, 2, 6, 64, 128, 64
    _, offsets, tok, active = route(T, k, E, seed=2)
    parts = make(E, N, K, group, True, 1)
    W = native.q4_weights(*parts, group)
    x = rand((T, K), BF, 1)
    slots = torch.arange(E, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = active[1: 1 + int(active[0])].tolist()

    def call(slot_of, offsets, tok, active):
        out = torch.full((T * k, N), 7.0, dtype=F32, device="cuda")
        status.zero_()
        native.expert_linear_q4(W, slot_of.cuda(), x, T, E, k, offsets, tok, active, out, dev_status=status)
        return out, int(status)

    def check(out, skipped, zero=()):
        for e, r0, r1 in ranges(offsets):
            rows = x[tok[r0:r1].long()]
            for z in zero:
                if r0 <= z < r1:
                    rows[z - r0] = 0
            if e in skipped:
                assert (out[r0:r1] == 7).all()
            else:
                assert_close(out[r0:r1], *reference(parts, group, 0, e, rows))

    bad = slots.clone()
    bad[ids[0]], bad[ids[1]] = E, -2
    out, st = call(bad, offsets, tok, active)
    assert st == native.DEV_BAD_SLOT
    check(out, {ids[0], ids[1]})
    for value in (E, -1, 2 ** 31 - 1):                   # an id outside the experts
        act2 = active.clone()
        act2[2] = value
        out, st = call(slots, offsets, tok, act2)
        assert st == native.DEV_BAD_INDEX
        check(out, {ids[1]})
    for value in (-1, T, 2 ** 31 - 1):                   # a token outside the batch
        tok2 = tok.clone()
        tok2[3] = value
        out, st = call(slots, offsets, tok2, active)
        assert st == native.DEV_BAD_INDEX
        check(out, (), zero=(3,))
    off2 = offsets.clone()
    off2[E] = T * k + 1                                  # rows past the batch
    out, st = call(slots, off2, tok, active)
    assert st == native.DEV_BAD_INDEX
    check(out, {E - 1})
    act2 = active.clone()                                # a count past the list: no more than E entries are read
    act2[0] = 2 ** 31 - 1
    act2[1 + len(ids):] = -1
    out, st = call(slots, offsets, tok, act2)
    assert st == native.DEV_BAD_INDEX
    check(out, ())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_far_values(dtype):
    """Activations at the ends of their type's range, zero scales, an offset alone,
    and a NaN or infinity that stays in its row."""
    N, K, group = 64, 256, 64
    codes, scale, mn = make(1, N, K, group, True, 4)
    scale[0, :, 0] = 0                                   # a group that is its offset
    x = rand((6, K), dtype, 1)
    x[1] *= 2.0 ** -14
    x[2] *= 2.0 ** (100 if dtype == BF else 10)
    x[3] = 0
    x[4, 5] = float("nan")
    x[5, 70] = float("inf")
    out = torch.empty(6, N, dtype=F32, device="cuda")
    native.linear_q4(native.q4_weights(codes, scale, mn, group), 0, x, 6, out)
    y, tol = reference((codes, scale, mn), group, 0, 0, x[:4])
    assert_close(out[:4], y, tol)
    assert torch.isnan(out[4]).all() and not torch.isfinite(out[5]).any()


def test_scale_at_fp16_limit():
    """s = 65504 without offset: w = s*(q-8) reaches 524032, beyond fp16."""
    codes = torch.randint(0, 256, (1, 32, 32), generator=torch.Generator().manual_seed(1), dtype=torch.uint8).cuda()
    scale = torch.full((1, 32, 1), 65504.0, device="cuda").half()
    x = rand((3, 64), BF, 1)
    out = torch.empty(3, 32, dtype=F32, device="cuda")
    native.linear_q4(native.q4_weights(codes, scale, None, 64), 0, x, 3, out)
    assert_close(out, *reference((codes, scale, None), 64, 0, 0, x))


def test_streams_graphs_and_repeats():
    T, k, E, N, K, group = 16, 4, 24, 256, 512, 64
    _, offsets, tok, active = route(T, k, E, seed=6, crowd=0.5)
    parts = make(E, N, K, group, True, 7)
    W = native.q4_weights(*parts, group)
    slot_of = torch.arange(E, dtype=torch.int32, device="cuda")
    x = rand((T, K), BF, 1)
    out = torch.empty(T * k, N, dtype=BF, device="cuda")
    many = torch.empty(T, N, dtype=BF, device="cuda")

    def both():
        native.expert_linear_q4(W, slot_of, x, T, E, k, offsets, tok, active, out)
        native.linear_q4(W, 3, x, T, many)

    both()
    want = out.clone(), many.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        many.zero_()
        both()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(many, want[1])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both()
        graphs.append(g)
    for i in range(4):
        out.zero_()
        many.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(many, want[1])


def test_two_calls_at_once_and_bits():
    """Two streams with their own tensors; int16 tensors are bf16 bits."""
    T, N, K, group = 20, 512, 1024, 64
    sets = []
    for seed in (1, 2):
        parts = make(2, N, K, group, True, seed)
        sets.append((parts, native.q4_weights(*parts, group), rand((T, K), BF, seed),
                     [torch.empty(T, N // 2, dtype=BF, device="cuda") for _ in range(8)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(8):
        for _, W, x, outs, stream in sets:
            if i % 2:
                native.linear_q4(W, 1, x.view(torch.int16), T, outs[i].view(torch.int16), native.ACT_SWIGLU, stream)
            else:
                native.linear_q4(W, 1, x, T, outs[i], native.ACT_SWIGLU, stream)
    torch.cuda.synchronize()
    for parts, _, x, outs, _ in sets:
        assert_close(outs[0], *reference(parts, group, native.ACT_SWIGLU, 1, x))
        assert all(torch.equal(o, outs[0]) for o in outs)


def test_many_experts_and_rows():
    """As many experts as there may be, k = 16; and a batch of many passes."""
    T, k, E, N, K, group = 90, 16, 4096, 32, 64, 32
    _, offsets, tok, active = route(T, k, E, seed=3, crowd=0.4)
    parts = make(E, N, K, group, False, 5)
    slot_of = torch.arange(E - 1, -1, -1, dtype=torch.int32, device="cuda")
    x = rand((T, K), BF, 1)
    out = torch.empty(T * k, N, dtype=F32, device="cuda")
    native.expert_linear_q4(native.q4_weights(*parts, group), slot_of, x, T, E, k, offsets, tok, active, out)
    for e, r0, r1 in ranges(offsets)[::37] + ranges(offsets)[:1]:
        assert_close(out[r0:r1], *reference(parts, group, 0, E - 1 - e, x[tok[r0:r1].long()]))
    T = 1003
    parts = make(1, 96, 288, 32, True, 6)
    x, out = rand((T, 288), FP, 2), torch.empty(T, 96, dtype=FP, device="cuda")
    native.linear_q4(native.q4_weights(*parts, 32), 0, x, T, out)
    assert_close(out, *reference(parts, 32, 0, 0, x))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_outlier_in_a_row(dtype):
    """One value 2^20 times the others, its weights 0: the others keep their digits
    down to its share of the sums it passes through. Weights are formed as q and
    -8, so it adds 8 s x and takes 8 s x off again. Each product instruction of
    its group (4 of 16 k) aligns its 16 products and the sum so far to the largest
    of them and cuts below 2^-23 of it: 17 cuts each; scaling, the group's sum of
    x and the additions that join them round at most 8 times more. In all 76 times
    2^-23 of 8 s 2^12, 0.3 s, where the others' results are about 0.4 s; losing
    them to the outlier's own fp16 or bf16 step (2^12 * 2^-8 and more) is 16 s."""
    N, K, group = 64, 512, 64
    codes, scale, _ = make(1, N, K, group, False, 8)
    codes[0, :, 50] = 0x88                               # weights 100 and 101 are 0
    x = rand((3, K), dtype, 1, 2.0 ** -8)
    x[:, 100] = 2.0 ** 12
    out = torch.empty(3, N, dtype=F32, device="cuda")
    native.linear_q4(native.q4_weights(codes, scale, None, group), 0, x, 3, out)
    x0 = x.clone()
    x0[:, 100] = 0
    y, tol = reference((codes, scale, None), group, 0, 0, x0)
    s = scale[0, :, 1].double()
    assert_close(out, y, tol + 76 * 2.0 ** -23 * 8 * 2.0 ** 12 * s)


def test_codes_past_32_bit_offsets():
    slots, N, K, group = 66, 8192, 8192, 128            # 2.2e9 bytes of codes
    codes = torch.randint(0, 256, (slots, N, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.full((slots, N, K // group), 2.0 ** -9, dtype=FP, device="cuda")
    x = rand((2, K), BF, 1)
    out = torch.empty(2, N, dtype=BF, device="cuda")
    native.linear_q4(native.q4_weights(codes, scale, None, group), slots - 1, x, 2, out)
    W, mag = dense(codes[slots - 1], scale[slots - 1], None, group)
    assert_close(out, x.double() @ W.t(), (x.double().abs() @ mag.t()) * bound(K, group))


def test_far_gate_of_a_large_up_row():
    """exp(-gate) beyond fp32, the up row large enough for a result near one."""
    # Gate -8 s x_0 and up 2^14 x_128 are exact. exp is off by two steps of 2^-24 and, at 2^-130 with 2^-149 the
    # smallest subnormal, by 2^-20; two more roundings: below 2^-19 together.
    gate_scale = torch.tensor([11.0, 11.0625, 11.125, 11.1875, 11.25, 11.0, 11.125, 11.25])
    codes = torch.full((64, 128), 0x88, dtype=torch.uint8)
    codes[:32, 0], codes[32:, 64] = 0x80, 0x89
    scale = torch.zeros(64, 2)
    scale[:32, 0], scale[32:, 1] = gate_scale.repeat(4), 2.0 ** 14
    x = torch.zeros(1, 256, dtype=BF)
    x[0, 0], x[0, 128] = 1.0, 2.0 ** 112
    out = torch.empty(1, 32, dtype=F32, device="cuda")
    native.linear_q4(native.q4_weights(codes.cuda(), scale.half().cuda(), None, 128), 0, x.cuda(), 1, out,
                     native.ACT_SWIGLU)
    want = (silu(-8 * gate_scale.double().repeat(4)) * 2.0 ** 126).cuda()[None]
    assert (want.abs() > 1).all()
    assert_close(out, want, want.abs() * 2.0 ** -19)
