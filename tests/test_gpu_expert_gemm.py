"""Unquantised expert products, their gradients, and SwiGLU, against the
formulas in 64 bits."""
import pytest
import torch

from bit_expert_ffn_fp32_b200 import native
from routed import assert_close, ranges, route, silu, sum_bound

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def forward(a, W, T, k, offsets, tok, out, status=None, stream=None):
    E, N, K = W.shape
    native.expert_gemm(a, W, T, E, k, N, K, offsets, tok, out, dev_status=status, stream=stream)


def forward_ref(a, W, offsets, tok):
    E, N, K = W.shape
    P = tok.numel() if tok is not None else a.shape[0]
    y = torch.zeros(P, N, dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(y)
    for e, r0, r1 in ranges(offsets):
        x = (a[tok[r0:r1].long()] if tok is not None else a[r0:r1]).double()
        y[r0:r1] = x @ W[e].double().t()
        mag[r0:r1] = x.abs() @ W[e].double().abs().t()
    return y, mag * sum_bound(K)


def dgrad_ref(dy, W, offsets):
    E, N, K = W.shape
    y = torch.zeros(dy.shape[0], K, dtype=torch.float64, device=dy.device)
    mag = torch.zeros_like(y)
    for e, r0, r1 in ranges(offsets):
        y[r0:r1] = dy[r0:r1].double() @ W[e].double()
        mag[r0:r1] = dy[r0:r1].double().abs() @ W[e].double().abs()
    return y, mag * sum_bound(N)


def wgrad_ref(dy, a, E, offsets, tok, base=None):
    N, K = dy.shape[1], a.shape[1]
    y = torch.zeros(E, N, K, dtype=torch.float64, device=dy.device) if base is None else base.double()
    tol = y.abs() * 2.0 ** -24
    for e, r0, r1 in ranges(offsets):
        x = (a[tok[r0:r1].long()] if tok is not None else a[r0:r1]).double()
        y[e] += dy[r0:r1].double().t() @ x
        tol[e] += dy[r0:r1].double().abs().t() @ x.abs() * sum_bound(r1 - r0)
    return y, tol + y.abs() * 2.0 ** -24


# T, k, E, N, K, share of tokens on expert 0: one token; fewer rows than a tile, odd counts; a crowded expert of
# several tiles; N and K below, beside and past the tile edges; the tiny layer; one expert for every row
SHAPES = [
    (1, 1, 1, 8, 8, 0.0),
    (1, 4, 16, 64, 72, 0.0),
    (7, 2, 5, 136, 200, 0.5),
    (33, 3, 8, 128, 64, 1.0),
    (333, 4, 64, 512, 512, 0.3),
    (601, 2, 6, 264, 328, 0.9),
    (1000, 1, 1, 392, 1096, 0.0),
    (257, 16, 300, 256, 136, 0.1),
    (64, 10, 512, 1536, 256, 0.0),
    (300, 16, 4096, 64, 192, 0.5),   # as many experts as there may be
]


@pytest.mark.parametrize("T,k,E,N,K,crowd", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype,gather", [(BF, BF, True), (FP, F32, False), (BF, F32, True), (FP, FP, False)])
def test_forward(T, k, E, N, K, crowd, dtype, out_dtype, gather):
    _, offsets, tok, _ = route(T, k, E, seed=T + E, crowd=crowd)
    P = T * k
    a = rand((T if gather else P, K), dtype, 1)
    W = rand((E, N, K), dtype, 2, K ** -0.5)
    out = torch.full((P, N), float("nan"), dtype=out_dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    forward(a, W, T, k, offsets, tok if gather else None, out, status)
    assert_close(out, *forward_ref(a, W, offsets, tok if gather else None))
    assert int(status) == 0


@pytest.mark.parametrize("T,k,E,N,K,crowd", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (FP, F32)])
def test_dgrad(T, k, E, N, K, crowd, dtype, out_dtype):
    _, offsets, _, _ = route(T, k, E, seed=T + E, crowd=crowd)
    dy = rand((T * k, N), dtype, 3)
    W = rand((E, N, K), dtype, 2, N ** -0.5)
    da = torch.full((T * k, K), float("nan"), dtype=out_dtype, device="cuda")
    native.expert_gemm_dgrad(dy, W, T, E, k, N, K, offsets, da)
    assert_close(da, *dgrad_ref(dy, W, offsets))


@pytest.mark.parametrize("T,k,E,N,K,crowd", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype,gather,base", [(BF, BF, True, False), (FP, F32, False, True),
                                                         (BF, F32, True, True), (FP, FP, False, False),
                                                         (BF, BF, False, True)])
def test_wgrad(T, k, E, N, K, crowd, dtype, out_dtype, gather, base):
    _, offsets, tok, _ = route(T, k, E, seed=T + E, crowd=crowd)
    P = T * k
    dy = rand((P, N), dtype, 3)
    a = rand((T if gather else P, K), dtype, 1)
    b = rand((E, N, K), out_dtype, 4) if base else None
    dW = torch.full((E, N, K), float("nan"), dtype=out_dtype, device="cuda")
    native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok if gather else None, dW, base=b)
    ref = wgrad_ref(dy, a, E, offsets, tok if gather else None, b)
    assert_close(dW, *ref)
    if base:   # in place
        native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok if gather else None, b, base=b)
        assert torch.equal(b, dW)


def test_gradients_against_differences():
    """dot(dy, f(a + h v) - f(a - h v)) = 2 h dot(da, v), and the same for W: the
    product is linear in each, so differences of the formula are exact up to its
    sums; the gradients are compared at the size of their own error."""
    T, k, E, N, K = 40, 3, 7, 72, 88
    _, offsets, tok, _ = route(T, k, E, seed=5, crowd=0.4)
    P = T * k
    a, W, dy = rand((P, K), BF, 1), rand((E, N, K), BF, 2), rand((P, N), BF, 3)
    v, V = rand((P, K), BF, 4), rand((E, N, K), BF, 5)
    da = torch.empty(P, K, dtype=F32, device="cuda")
    dW = torch.empty(E, N, K, dtype=F32, device="cuda")
    native.expert_gemm_dgrad(dy, W, T, E, k, N, K, offsets, da)
    native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, None, dW)

    def f(a, W):
        y = torch.zeros(P, N, dtype=torch.float64, device="cuda")
        for e, r0, r1 in ranges(offsets):
            y[r0:r1] = a[r0:r1] @ W[e].t()
        return (y * dy.double()).sum()

    h = 2.0 ** -6
    a, W, v, V = a.double(), W.double(), v.double(), V.double()
    diff_a = (f(a + h * v, W) - f(a - h * v, W)) / (2 * h)
    diff_W = (f(a, W + h * V) - f(a, W - h * V)) / (2 * h)
    tol_a = (dgrad_ref(dy, W, offsets)[1] * v.abs()).sum() + 1e-9 * diff_a.abs()
    tol_W = (wgrad_ref(dy, a, E, offsets, None)[1] * V.abs()).sum() + 1e-9 * diff_W.abs()
    assert (diff_a - (da.double() * v).sum()).abs() <= tol_a
    assert (diff_W - (dW.double() * V).sum()).abs() <= tol_W


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_in_their_expert(bad):
    """Rows, weights and columns next to a tile's ragged edge never reach another
    expert's result: not as a product with a zero either."""
    T, k, E, N, K = 90, 2, 9, 136, 200
    _, offsets, tok, _ = route(T, k, E, seed=3)
    P = T * k
    a, W, dy = rand((P, K), BF, 1), rand((E, N, K), BF, 2, K ** -0.5), rand((P, N), BF, 3)
    o = offsets.tolist()
    out, da = torch.empty(P, N, dtype=BF, device="cuda"), torch.empty(P, K, dtype=BF, device="cuda")
    dW = torch.empty(E, N, K, dtype=F32, device="cuda")
    for e in (0, 4, 8):
        a2, W2, dy2 = a.clone(), W.clone(), dy.clone()
        a2[o[e]:o[e + 1]] = bad
        dy2[o[e]:o[e + 1]] = bad
        W2[e] = bad
        ref = [torch.empty_like(t) for t in (out, da, dW)]
        for aa, ww, dd, (y, x, w) in ((a, W, dy, ref), (a2, W2, dy2, (out, da, dW))):
            native.expert_gemm(aa, ww, T, E, k, N, K, offsets, None, y)
            native.expert_gemm_dgrad(dd, ww, T, E, k, N, K, offsets, x)
            native.expert_gemm_wgrad(dd, aa, T, E, k, N, K, offsets, None, w)
        keep = torch.ones(P, dtype=torch.bool, device="cuda")
        keep[o[e]:o[e + 1]] = False
        others = [i for i in range(E) if i != e]
        assert torch.equal(out[keep], ref[0][keep]) and torch.equal(da[keep], ref[1][keep])
        assert torch.equal(dW[others], ref[2][others])
        assert not torch.isfinite(out[~keep].float()).any() and not torch.isfinite(dW[e]).any()


def test_rows_outside_the_experts_are_left():
    T, k, E, N, K = 50, 2, 4, 72, 64
    P = T * k
    offsets = torch.tensor([3, 3, 41, 60, 90], dtype=torch.int32, device="cuda")
    a, W, dy = rand((P, K), BF, 1), rand((E, N, K), BF, 2), rand((P, N), BF, 3)
    out = torch.full((P, N), 7.0, dtype=F32, device="cuda")
    da = torch.full((P, K), 7.0, dtype=F32, device="cuda")
    dW = torch.full((E, N, K), 7.0, dtype=F32, device="cuda")
    native.expert_gemm(a, W, T, E, k, N, K, offsets, None, out)
    native.expert_gemm_dgrad(dy, W, T, E, k, N, K, offsets, da)
    native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, None, dW)
    for got, ref in ((out, forward_ref(a, W, offsets, None)), (da, dgrad_ref(dy, W, offsets))):
        assert torch.equal(got[:3], torch.full_like(got[:3], 7)) and torch.equal(got[90:], torch.full_like(got[90:], 7))
        assert_close(got[3:90], ref[0][3:90], ref[1][3:90])
    assert_close(dW, *wgrad_ref(dy, a, E, offsets, None))
    assert (dW[0] == 0).all()


def test_bad_tables_are_flagged_and_skipped():
    T, k, E, N, K = 20, 2, 3, 64, 64
    P = T * k
    a, W, dy = rand((P, K), BF, 1), rand((E, N, K), BF, 2), rand((P, N), BF, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for table in ([0, 10, 5, 40], [0, 10, 20, 41], [-1, 10, 20, 40], [0, 2 ** 31 - 1, 20, 40]):
        offsets = torch.tensor(table, dtype=torch.int32, device="cuda")
        good = [e for e in range(E) if 0 <= table[e] <= table[e + 1] <= P]
        out = torch.full((P, N), 7.0, dtype=F32, device="cuda")
        da = torch.full((P, K), 7.0, dtype=F32, device="cuda")
        dW = torch.full((E, N, K), 7.0, dtype=F32, device="cuda")
        for call in (lambda: native.expert_gemm(a, W, T, E, k, N, K, offsets, None, out, dev_status=status),
                     lambda: native.expert_gemm_dgrad(dy, W, T, E, k, N, K, offsets, da, dev_status=status),
                     lambda: native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, None, dW, dev_status=status)):
            status.zero_()
            call()
            assert int(status) == native.DEV_BAD_INDEX
        claims = torch.zeros(P, dtype=torch.int32)           # a row that two experts claim holds either's values
        for e in good:
            claims[table[e]:table[e + 1]] += 1
        rows, once = claims > 0, (claims == 1).cuda()
        for e in good:
            r0, r1 = table[e], table[e + 1]
            y = a[r0:r1].double() @ W[e].double().t()
            tol = (a[r0:r1].double().abs() @ W[e].double().abs().t()) * sum_bound(K)
            at = once[r0:r1]
            assert_close(out[r0:r1][at], y[at], tol[at])
        assert (out[~rows.cuda()] == 7).all() and (da[~rows.cuda()] == 7).all()
        for e in set(range(E)) - set(good):
            assert (dW[e] == 0).all()


def test_bad_tokens_count_as_zeros():
    T, k, E, N, K = 30, 2, 4, 136, 72
    P = T * k
    _, offsets, tok, _ = route(T, k, E, seed=9)
    a, W, dy = rand((T, K), BF, 1), rand((E, N, K), BF, 2), rand((P, N), BF, 3)
    bad = tok.clone()
    bad[5], bad[17], bad[P - 1] = -1, T, 2 ** 31 - 1
    a0 = a[tok.long()]
    a0[[5, 17, P - 1]] = 0
    out, dW = torch.empty(P, N, dtype=BF, device="cuda"), torch.empty(E, N, K, dtype=F32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    native.expert_gemm(a, W, T, E, k, N, K, offsets, bad, out, dev_status=status)
    assert int(status) == native.DEV_BAD_INDEX
    assert_close(out, *forward_ref(a0, W, offsets, None))
    status.zero_()
    native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, bad, dW, dev_status=status)
    assert int(status) == native.DEV_BAD_INDEX
    assert_close(dW, *wgrad_ref(dy, a0, E, offsets, None))


def test_no_tokens():
    E, N, K = 5, 72, 64
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    W = rand((E, N, K), BF, 1)
    none = torch.empty(0, K, dtype=BF, device="cuda")
    out = torch.full((4, N), 7.0, dtype=BF, device="cuda")
    native.expert_gemm(none, W, 0, E, 2, N, K, offsets, None, out)
    dW, base = torch.full((E, N, K), 7.0, dtype=BF, device="cuda"), rand((E, N, K), BF, 2)
    native.expert_gemm_wgrad(torch.empty(0, N, dtype=BF, device="cuda"), none, 0, E, 2, N, K, offsets, None, dW)
    assert (out == 7).all() and (dW == 0).all()
    native.expert_gemm_wgrad(torch.empty(0, N, dtype=BF, device="cuda"), none, 0, E, 2, N, K, offsets, None, dW,
                             base=base)
    assert torch.equal(dW, base)


def test_weights_past_32_bit_offsets():
    T, k, E, N, K = 3, 4, 130, 8192, 2048           # 2.18e9 weights
    W = torch.empty(E, N, K, dtype=BF, device="cuda").normal_(std=K ** -0.5)
    a = rand((T, K), BF, 1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = 2                                  # expert 0 has two rows, the last two have five each
    offsets[E - 1], offsets[E] = 7, 12
    tok = torch.tensor([0, 1, 2, 0, 1, 2, 0, 1, 2, 0, 1, 2], dtype=torch.int32, device="cuda")
    out = torch.empty(T * k, N, dtype=BF, device="cuda")
    forward(a, W, T, k, offsets, tok, out)
    assert_close(out, *forward_ref(a, W, offsets, tok))


def test_streams_graphs_and_repeats():
    """A side stream, two captured graphs replayed in turn, and equal bits from equal calls."""
    T, k, E, N, K = 200, 4, 16, 256, 192
    _, offsets, tok, _ = route(T, k, E, seed=8, crowd=0.5)
    P = T * k
    a, W, dy = rand((T, K), BF, 1), rand((E, N, K), BF, 2), rand((P, N), BF, 3)
    out, da = torch.empty(P, N, dtype=BF, device="cuda"), torch.empty(P, K, dtype=BF, device="cuda")
    dW = torch.empty(E, N, K, dtype=F32, device="cuda")

    def all_three():
        native.expert_gemm(a, W, T, E, k, N, K, offsets, tok, out)
        native.expert_gemm_dgrad(dy, W, T, E, k, N, K, offsets, da)
        native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok, dW)

    all_three()
    want = [t.clone() for t in (out, da, dW)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for t in (out, da, dW):
            t.zero_()
        all_three()
    torch.cuda.synchronize()
    assert all(torch.equal(t, w) for t, w in zip((out, da, dW), want))
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_three()
        graphs.append(g)
    for i in range(6):
        for t in (out, da, dW):
            t.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip((out, da, dW), want))
    # the tables are read at replay: another routing through the same graph
    _, offsets2, tok2, _ = route(T, k, E, seed=81)
    offsets.copy_(offsets2)
    tok.copy_(tok2)
    graphs[0].replay()
    assert_close(out, *forward_ref(a, W, offsets, tok))


def test_two_calls_at_once():
    """Two streams with their own tensors, many calls in flight on both."""
    T, k, E, N, K = 300, 4, 12, 256, 320
    sets = []
    for seed in (1, 2):
        _, offsets, tok, _ = route(T, k, E, seed=seed, crowd=0.3)
        a, W, dy = rand((T, K), BF, seed), rand((E, N, K), BF, seed + 10), rand((T * k, N), BF, seed + 20)
        outs = [(torch.empty(T * k, N, dtype=BF, device="cuda"), torch.empty(T * k, K, dtype=BF, device="cuda"),
                 torch.empty(E, N, K, dtype=F32, device="cuda")) for _ in range(6)]
        sets.append((offsets, tok, a, W, dy, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(6):
        for offsets, tok, a, W, dy, outs, stream in sets:
            native.expert_gemm(a, W, T, E, k, N, K, offsets, tok, outs[i][0], stream=stream)
            native.expert_gemm_dgrad(dy, W, T, E, k, N, K, offsets, outs[i][1], stream=stream)
            native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok, outs[i][2], stream=stream)
    torch.cuda.synchronize()
    for offsets, tok, a, W, dy, outs, _ in sets:
        assert_close(outs[0][0], *forward_ref(a, W, offsets, tok))
        assert_close(outs[0][1], *dgrad_ref(dy, W, offsets))
        assert_close(outs[0][2], *wgrad_ref(dy, a, E, offsets, tok))
        for o in outs[1:]:
            assert all(torch.equal(x, y) for x, y in zip(o, outs[0]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sum_in_place_through_a_graph(dtype):
    """Three replays add three times; integers, so that no sum is rounded."""
    T, k, E, N, K = 40, 2, 8, 72, 136
    _, offsets, tok, _ = route(T, k, E, seed=4, crowd=0.3)
    g = torch.Generator().manual_seed(1)
    dy = torch.randint(-1, 2, (T * k, N), generator=g).to(BF).cuda()
    a = torch.randint(-1, 2, (T, K), generator=g).to(BF).cuda()
    dW = torch.zeros(E, N, K, dtype=dtype, device="cuda")
    native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok, dW)
    once = dW.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok, dW, base=dW)
    for _ in range(2):
        graph.replay()
    assert torch.equal(dW, 3 * once) and torch.equal(once.double(), wgrad_ref(dy, a, E, offsets, tok)[0])


@pytest.mark.parametrize("dtype,separate", [(BF, True), (BF, False), (F32, True), (F32, False)])
def test_non_finite_sum_stays_in_its_place(dtype, separate):
    T, k, E, N, K = 50, 2, 5, 72, 136
    _, offsets, tok, _ = route(T, k, E, seed=4)
    dy, a = rand((T * k, N), BF, 1), rand((T, K), BF, 2)
    base = rand((E, N, K), dtype, 3)
    dW = torch.empty_like(base)
    native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok, dW, base=base)
    spots = [(0, 0, 0), (1, 5, 77), (4, N - 1, K - 1)]
    for i, s in enumerate(spots):
        base[s] = float("nan") if i % 2 else float("inf")
    out = torch.empty_like(base) if separate else base
    native.expert_gemm_wgrad(dy, a, T, E, k, N, K, offsets, tok, out, base=base)
    ok = torch.ones(E, N, K, dtype=torch.bool, device="cuda")
    for s in spots:
        ok[s] = False
        assert not torch.isfinite(out[s])
    assert torch.equal(out[ok], dW[ok])


def test_bf16_bits_and_overflow():
    """int16 tensors are bf16 bits; results past fp16 become infinities of their sign."""
    T, k, E, N, K = 9, 2, 4, 64, 64
    _, offsets, tok, _ = route(T, k, E, seed=4)
    a, W = rand((T, K), BF, 1), rand((E, N, K), BF, 2)
    out, bits = torch.empty(T * k, N, dtype=BF, device="cuda"), torch.empty(T * k, N, dtype=torch.int16, device="cuda")
    forward(a, W, T, k, offsets, tok, out)
    native.expert_gemm(a.view(torch.int16), W.view(torch.int16), T, E, k, N, K, offsets, tok, bits)
    assert torch.equal(bits.view(BF), out)
    big = torch.full((T, K), 200.0, dtype=FP, device="cuda")
    Wb = torch.full((E, N, K), 100.0, dtype=FP, device="cuda")
    Wb[:, 1::2] = -100.0
    o = torch.empty(T * k, N, dtype=FP, device="cuda")
    forward(big, Wb, T, k, offsets, tok, o)
    assert (o[:, ::2] == float("inf")).all() and (o[:, 1::2] == -float("inf")).all()


# ------------------------------------------------------------------ SwiGLU
def swiglu_ref(gu, dh=None):
    f = gu.shape[1] // 2
    g, u = gu[:, :f].double(), gu[:, f:].double()
    s = torch.special.expit(g)
    if dh is None:
        return g * s * u
    dh = dh.double()
    return torch.cat((dh * u * (s + g * s * torch.special.expit(-g)), dh * g * s), dim=1)


@pytest.mark.parametrize("rows,f", [(1, 8), (3, 72), (7, 256), (1000, 768), (333, 1096), (5, 16384)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_swiglu(rows, f, dtype):
    # a few fp32 roundings of the terms: 2^-18 of their magnitude is far above them
    gu, dh = rand((rows, 2 * f), dtype, 1, 2.0), rand((rows, f), dtype, 2)
    h, dgu = torch.empty(rows, f, dtype=dtype, device="cuda"), torch.empty(rows, 2 * f, dtype=dtype, device="cuda")
    native.swiglu(gu, rows, f, h)
    want = swiglu_ref(gu)
    assert_close(h, want, want.abs() * 2.0 ** -18)
    native.swiglu_backward(gu, dh, rows, f, dgu)
    want = swiglu_ref(gu, dh)
    g, u, d = gu[:, :f].double().abs(), gu[:, f:].double().abs(), dh.double().abs()
    mag = torch.cat((d * u * (1 + g), d * g), dim=1)
    assert_close(dgu, want, mag * 2.0 ** -20)
    native.swiglu_backward(gu, dh, rows, f, gu)      # in place
    assert torch.equal(gu, dgu)


def test_swiglu_gradient_against_differences():
    gu, dh = rand((20, 48), BF, 1), rand((20, 24), BF, 2)
    dgu = torch.empty_like(gu)
    native.swiglu_backward(gu, dh, 20, 24, dgu)
    h = 1e-5
    v = rand((20, 48), BF, 3).double()
    up, down = (silu(t[:, :24]) * t[:, 24:] for t in (gu.double() + h * v, gu.double() - h * v))
    diff = ((up - down) / (2 * h) * dh.double()).sum()
    # each gradient is rounded to bf16 once; differences are off by h^2 times a third derivative below 10
    tol = (dgu.double().abs() * v.abs()).sum() * 2.0 ** -8 + 1e-6 * v.abs().sum()
    assert (diff - (dgu.double() * v).sum()).abs() <= tol


def test_swiglu_far_values():
    """Saturated gates: exactly u * g or a vanishing product, never NaN."""
    g = torch.tensor([[-3e38, -200.0, -95.0, -88.0, 88.0, 200.0, 3e38, 0.0]], device="cuda")
    gu = torch.cat((g, torch.ones_like(g)), dim=1).to(BF)
    h, dgu = torch.empty(1, 8, dtype=BF, device="cuda"), torch.empty(1, 16, dtype=BF, device="cuda")
    native.swiglu(gu, 1, 8, h)
    native.swiglu_backward(gu, torch.ones(1, 8, dtype=BF, device="cuda"), 1, 8, dgu)
    want, dwant = swiglu_ref(gu), swiglu_ref(gu, torch.ones(1, 8, device="cuda"))
    # products below fp32's normal range may be flushed: 88 * 2^-126 at most
    assert_close(h, want, want.abs() * 2.0 ** -18 + 2.0 ** -119)
    assert_close(dgu, dwant, dwant.abs() * 2.0 ** -18 + 2.0 ** -119)


def test_swiglu_far_gate_of_a_large_product():
    """exp(-g) beyond fp32's largest power of two: the product with a large u is
    not far from one, so sig(g) may not vanish on the way."""
    # exp(g), g = -90..-87.5: its argument in powers of two (130) is off by 2^-17 + 2^-18, exp by 0.7 of that; the
    # subnormal exp of 2^-130 keeps 19 bits; together below 2^-15.9, a few roundings of 2^-24 on top
    g = torch.tensor([[-87.5, -88.0, -88.5, -88.75, -89.0, -89.25, -89.5, -90.0]], device="cuda").to(BF)
    u = torch.full_like(g, 2.0 ** 124)
    gu, dh = torch.cat((g, u), dim=1), torch.full_like(g, 2.0 ** 1)
    h, dgu = torch.empty(1, 8, dtype=BF, device="cuda"), torch.empty(1, 16, dtype=BF, device="cuda")
    native.swiglu(gu, 1, 8, h)
    native.swiglu_backward(gu, dh, 1, 8, dgu)
    want, dwant = swiglu_ref(gu), swiglu_ref(gu, dh)
    assert (want.abs() > 0.1).all()
    assert_close(h, want, want.abs() * 2.0 ** -15)
    assert_close(dgu, dwant, dwant.abs() * 2.0 ** -15)
