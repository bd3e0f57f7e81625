"""Measured calls of the operators beside the block-quantised expert FFN:

  q4        products with 4-bit weights and group scales, dense (one matrix)
            or grouped by expert, optionally with the SwiGLU of the two row
            halves in the same pass
  gemm      unquantised products grouped by expert:  out[s] = W[e(s)] a[s]
  dgrad     their gradient to the rows:              da[s]  = W[e(s)]^T dy[s]
  wgrad     their gradient to the weights:           dW[e]  = sum_s dy[s] a[s]^T
  swiglu    h = silu(g) * u of rows [g | u], and its gradient

Rows are (token, expert) pairs in sorted order, as moe_permute leaves them:
expert e owns rows offsets[e] .. offsets[e+1]; sorted_tok names each row's token.

run(state) computes the plain form (elementary torch operations in 32 bits,
rounded once at the end), or, with ``own`` true, calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    """Twelve cases; d = 2048, f = 768, 512 experts, top-10 is the decoder layer of the
    workload table, d = 512, f = 256, 64 experts, top-4 its tiny layer."""
    return [
        # one decoded token through its ten experts' gate and up rows, SwiGLU in the same pass
        {"name": "q4_gate_up_T1", "op": "q4", "T": 1, "k": 10, "E": 512, "N": 1536, "K": 2048, "group": 64,
         "min": True, "swiglu": True, "gather": True, "skew": 0.0, "dtype": "bf16", "out": "bf16"},
        # the verify batch of one token and three drafts, down rows, written in fp32 for the combine
        {"name": "q4_down_T4", "op": "q4", "T": 4, "k": 10, "E": 512, "N": 2048, "K": 768, "group": 32,
         "min": False, "swiglu": False, "gather": False, "skew": 0.0, "dtype": "bf16", "out": "fp32"},
        # a dense projection next to the layer for one token (E = 0: one matrix for every row)
        {"name": "q4_dense_T1", "op": "q4", "T": 1, "k": 1, "E": 0, "N": 8192, "K": 8192, "group": 128,
         "min": False, "swiglu": False, "gather": False, "skew": 0.0, "dtype": "fp16", "out": "fp16"},
        # a batch of an odd number of sequences through a pool of experts
        {"name": "q4_gate_up_T37", "op": "q4", "T": 37, "k": 10, "E": 512, "N": 1536, "K": 2048, "group": 64,
         "min": True, "swiglu": True, "gather": True, "skew": 1.0, "dtype": "bf16", "out": "bf16"},
        # a verify batch through unquantised down rows, fp32 for the combine
        {"name": "gemm_down_T4", "op": "gemm", "T": 4, "k": 10, "E": 512, "N": 2048, "K": 768, "gather": False,
         "skew": 0.0, "dtype": "bf16", "out": "fp32"},
        # a prompt chunk's gate and up rows, x read by token
        {"name": "gemm_gate_up_T8192", "op": "gemm", "T": 8192, "k": 10, "E": 512, "N": 1536, "K": 2048,
         "gather": True, "skew": 0.5, "dtype": "bf16", "out": "bf16"},
        # the tiny layer's gradient to the hidden rows, odd token count
        {"name": "dgrad_tiny_T333", "op": "dgrad", "T": 333, "k": 4, "E": 64, "N": 512, "K": 256, "skew": 1.0,
         "dtype": "fp16", "out": "fp16"},
        # a training batch's gradient to x's rows
        {"name": "dgrad_T4096", "op": "dgrad", "T": 4096, "k": 10, "E": 128, "N": 1536, "K": 2048, "skew": 0.5,
         "dtype": "bf16", "out": "bf16"},
        # the tiny layer's weight gradient, added to the fp32 sum of earlier batches
        {"name": "wgrad_tiny_T333", "op": "wgrad", "T": 333, "k": 4, "E": 64, "N": 512, "K": 512, "gather": True,
         "skew": 1.0, "accumulate": True, "dtype": "fp16", "out": "fp32"},
        # a training batch's weight gradient of the down rows
        {"name": "wgrad_T4096", "op": "wgrad", "T": 4096, "k": 10, "E": 128, "N": 2048, "K": 768, "gather": False,
         "skew": 0.5, "accumulate": False, "dtype": "bf16", "out": "bf16"},
        # the activation of a prompt chunk's pairs, and its gradient for a training batch
        {"name": "swiglu_T8192", "op": "swiglu", "rows": 81920, "f": 768, "backward": False, "dtype": "bf16"},
        {"name": "swiglu_bwd_T4096", "op": "swiglu", "rows": 40960, "f": 768, "backward": True, "dtype": "fp16"},
    ]


def _log(rng, lo, hi, step=1):
    """An integer multiple of step, spread over the logarithm of [lo, hi]."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["q4", "q4", "gemm", "dgrad", "wgrad", "swiglu"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "swiglu":
        return {"op": op, "rows": _log(rng, 1, 81920), "f": _log(rng, 64, 1024, 8), "backward": rng.random() < 0.5,
                "dtype": dtype}
    if op == "q4":
        dense = rng.random() < 0.4
        group = rng.choice([32, 64, 128])
        return {"op": op, "T": _log(rng, 1, 64), "k": 1 if dense else rng.randint(1, 10),
                "E": 0 if dense else _log(rng, 16, 512), "N": _log(rng, 256, 8192 if dense else 2048, 32),
                "K": _log(rng, 256, 8192 if dense else 2048, group), "group": group, "min": rng.random() < 0.5,
                "swiglu": rng.random() < 0.5, "gather": not dense and rng.random() < 0.5,
                "skew": rng.choice([0.0, 0.5, 1.0]), "dtype": dtype, "out": rng.choice([dtype, "fp32"])}
    case = {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, 10), "E": _log(rng, 16, 128),
            "N": _log(rng, 64, 2048, 8), "K": _log(rng, 64, 2048, 8), "skew": rng.choice([0.0, 0.5, 1.0]),
            "dtype": dtype, "out": rng.choice([dtype, "fp32"])}
    if op != "dgrad":
        case["gather"] = rng.random() < 0.5
    if op == "wgrad":
        case["accumulate"] = rng.random() < 0.5
    return case


def _active(case):
    """Experts with at least one row, on average, under even routing."""
    T, k, E = case["T"], case["k"], case["E"]
    return 1 if E == 0 else E * (1 - (1 - k / E) ** T)


def work(case):
    if case["op"] == "swiglu":
        n = case["rows"] * case["f"]
        # forward: g, u in, h out; backward: g, u, dh in, dg, du out
        return {"bytes": n * 2 * (5 if case["backward"] else 3), "flops": n * (12 if case["backward"] else 5)}
    T, k, N, K = case["T"], case["k"], case["N"], case["K"]
    P, size = T * k, {"bf16": 2, "fp16": 2, "fp32": 4}
    i, o, A = size[case["dtype"]], size[case["out"]], _active(case)
    rows_in = (T if case.get("gather") else P) * K * i
    flops = 2 * P * N * K
    if case["op"] == "q4":
        w = A * N * K * (0.5 + (4 if case["min"] else 2) / case["group"])
        return {"bytes": w + rows_in + P * N * o // (2 if case["swiglu"] else 1), "flops": flops}
    if case["op"] == "gemm":
        return {"bytes": A * N * K * i + rows_in + P * N * o, "flops": flops}
    if case["op"] == "dgrad":
        return {"bytes": A * N * K * i + P * N * i + P * K * o, "flops": flops}
    # every expert's gradient is written, zeros or the earlier sum among them
    dw = case["E"] * N * K * o * (2 if case["accumulate"] else 1)
    return {"bytes": P * N * i + rows_in + dw, "flops": flops}


def _routing(case, rnd, dev):
    """Top-k routing of T tokens over E experts whose popularity spreads with skew, and its sorted order."""
    T, k, E = case["T"], case["k"], case["E"]
    if E == 0:
        return {"P": T}
    logits = torch.randn(T, E, generator=rnd, device=dev)
    logits += case["skew"] * torch.randn(E, generator=rnd, device=dev)
    idx = torch.sort(torch.topk(logits, k, dim=1).indices, dim=1).values
    order = torch.sort(idx.reshape(-1), stable=True)
    counts = torch.bincount(order.values, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = torch.cumsum(counts, 0)
    ids = torch.nonzero(counts).reshape(-1)
    active = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    active[0] = ids.numel()
    active[1: 1 + ids.numel()] = ids
    return {"P": T * k, "offsets": offsets, "sorted_tok": (order.indices // k).to(torch.int32), "active": active,
            "ids": ids, "most": int(counts.max())}


def prepare(case, seed):
    dev = torch.device("cuda")
    rnd = torch.Generator(device=dev)
    rnd.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=rnd, device=dev, dtype=dt)  # noqa: E731
    dt = DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] == "swiglu":
        state["gu"] = normal(case["rows"], 2 * case["f"])
        if case["backward"]:
            state["dh"] = normal(case["rows"], case["f"])
            state["out"] = torch.empty_like(state["gu"])
        else:
            state["out"] = torch.empty(case["rows"], case["f"], dtype=dt, device=dev)
        return state
    r = _routing(case, rnd, dev)
    state |= r
    T, k, E, N, K, P = case["T"], case["k"], case["E"], case["N"], case["K"], r["P"]
    out_dt = DTYPES[case["out"]]
    if case["op"] == "q4":
        # a pool with every expert resident, slots in another order than the experts
        S = max(E, 1)
        state["slot_of"] = torch.randperm(S, generator=rnd, device=dev).to(torch.int32)
        state["codes"] = torch.randint(0, 256, (S, N, K // 2), generator=rnd, device=dev, dtype=torch.uint8)
        unit = 1 / (4.6 * math.sqrt(K))  # 4.6: the standard deviation of a code
        state["scale"] = (unit * (0.5 + torch.rand(S, N, K // case["group"], generator=rnd, device=dev))).half()
        state["min"] = (-7.5 * state["scale"].float() * (0.8 + 0.4 * torch.rand(
            S, N, K // case["group"], generator=rnd, device=dev))).half() if case["min"] else None
        state["x"] = normal(T if case["gather"] else P, K)
        state["out"] = torch.empty(P, N // 2 if case["swiglu"] else N, dtype=out_dt, device=dev)
        if own:
            # the description of the pool that a program fills once
            from bit_expert_ffn_fp32_b200 import native
            state["weights"] = native.q4_weights(state["codes"], state["scale"], state["min"], case["group"])
        return state
    if case["op"] != "wgrad":
        state["W"] = normal(E, N, K) / math.sqrt(K if case["op"] == "gemm" else N)
    if case["op"] != "dgrad":
        state["a"] = normal(T if case["gather"] else P, K)
    if case["op"] != "gemm":
        state["dy"] = normal(P, N)
    if case["op"] == "wgrad":
        state["out"] = torch.zeros(E, N, K, dtype=out_dt, device=dev)
        if case["accumulate"]:
            state["before"] = torch.randn(E, N, K, generator=rnd, device=dev).to(out_dt)
    else:
        state["out"] = torch.empty(P, N if case["op"] == "gemm" else K, dtype=out_dt, device=dev)
    return state


def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from bit_expert_ffn_fp32_b200 import native
    c, out = s["case"], s["out"]
    if c["op"] == "swiglu":
        if c["backward"]:
            native.swiglu_backward(s["gu"], s["dh"], c["rows"], c["f"], out)
        else:
            native.swiglu(s["gu"], c["rows"], c["f"], out)
        return out
    T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
    if c["op"] == "q4":
        act = native.ACT_SWIGLU if c["swiglu"] else native.ACT_NONE
        if E == 0:
            native.linear_q4(s["weights"], 0, s["x"], T, out, act)
        else:
            native.expert_linear_q4(s["weights"], s["slot_of"], s["x"], T, E, k, s["offsets"],
                                    s["sorted_tok"] if c["gather"] else None, s["active"], out, act)
    elif c["op"] == "gemm":
        native.expert_gemm(s["a"], s["W"], T, E, k, N, K, s["offsets"], s["sorted_tok"] if c["gather"] else None, out)
    elif c["op"] == "dgrad":
        native.expert_gemm_dgrad(s["dy"], s["W"], T, E, k, N, K, s["offsets"], out)
    else:
        base = s["before"] if c["accumulate"] else None
        if base is not None and base.dtype == torch.float32:
            out = base  # an fp32 sum is added to in place
        native.expert_gemm_wgrad(s["dy"], s["a"], T, E, k, N, K, s["offsets"],
                                 s["sorted_tok"] if c["gather"] else None, out, base=base)
    return out


def _place(s):
    """Each row's place in a [active experts][most rows] grid."""
    offsets = s["offsets"].long()
    row = torch.arange(s["P"], device=offsets.device)
    first = offsets[s["ids"]]
    e = torch.searchsorted(first, row, right=True) - 1
    return e * s["most"] + row - first[e]


def _grid(rows, place, s):
    g = torch.zeros(s["ids"].numel() * s["most"], rows.shape[1], device=rows.device)
    g[place] = rows.float()
    return g.view(s["ids"].numel(), s["most"], -1)


def _dequant(s, slots):
    b = s["codes"][slots]
    q = torch.stack((b & 15, b >> 4), dim=-1).float().view(slots.numel(), s["case"]["N"], -1, s["case"]["group"])
    sc = s["scale"][slots].float().unsqueeze(-1)
    w = q * sc + s["min"][slots].float().unsqueeze(-1) if s["min"] is not None else (q - 8) * sc
    return w.view(slots.numel(), s["case"]["N"], -1)


def _silu_mul(g, u):
    return g / (1 + torch.exp(-g)) * u


def _plain(s):
    c, out = s["case"], s["out"]
    if c["op"] == "swiglu":
        g, u = s["gu"].float().split(c["f"], dim=1)
        if not c["backward"]:
            return _silu_mul(g, u).to(out.dtype)
        sig, dh = 1 / (1 + torch.exp(-g)), s["dh"].float()
        return torch.cat((dh * u * sig * (1 + g * (1 - sig)), dh * g * sig), dim=1).to(out.dtype)
    if c["op"] == "q4":
        if c["E"] == 0:
            y = s["x"].float() @ _dequant(s, s["slot_of"][:1].long())[0].t()
        else:
            place = _place(s)
            x = s["x"][s["sorted_tok"].long()] if c["gather"] else s["x"]
            W = _dequant(s, s["slot_of"][s["ids"]].long())
            y = torch.bmm(_grid(x, place, s), W.transpose(1, 2)).view(-1, c["N"])[place]
        return (_silu_mul(*y.split(c["N"] // 2, dim=1)) if c["swiglu"] else y).to(out.dtype)
    place = _place(s)
    if c["op"] == "gemm":
        a = s["a"][s["sorted_tok"].long()] if c["gather"] else s["a"]
        y = torch.bmm(_grid(a, place, s), s["W"][s["ids"]].float().transpose(1, 2))
        return y.view(-1, c["N"])[place].to(out.dtype)
    if c["op"] == "dgrad":
        da = torch.bmm(_grid(s["dy"], place, s), s["W"][s["ids"]].float())
        return da.view(-1, c["K"])[place].to(out.dtype)
    a = s["a"][s["sorted_tok"].long()] if c["gather"] else s["a"]
    d = torch.bmm(_grid(s["dy"], place, s).transpose(1, 2), _grid(a, place, s))
    dW = s["before"].float() if c["accumulate"] else torch.zeros(c["E"], c["N"], c["K"], device=d.device)
    dW[s["ids"]] += d
    return dW.to(out.dtype)


def exact(case, seed):
    """The same outputs in 64 bits, expert by expert from the definition."""
    s = prepare(case, seed)
    c = case
    if c["op"] == "swiglu":
        gu = s["gu"].double()
        g, u = gu[:, : c["f"]], gu[:, c["f"]:]
        if not c["backward"]:
            return torch.special.expit(g) * g * u
        # d silu(g) = sigmoid(g) + silu(g) (1 - sigmoid(g))
        dh, sg = s["dh"].double(), torch.special.expit(g)
        d = torch.empty_like(gu)
        d[:, : c["f"]] = dh * u * (sg + g * sg * torch.special.expit(-g))
        d[:, c["f"]:] = dh * g * sg
        return d
    if c["op"] == "q4" and c["E"] == 0:
        off = [0, c["T"]]
    else:
        off = s["offsets"].tolist()
    tok = s["sorted_tok"].long() if c.get("gather") else None
    experts = [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e] < off[e + 1]]
    if c["op"] == "wgrad":
        dW = s["before"].double() if c["accumulate"] else torch.zeros(s["out"].shape, dtype=torch.float64,
                                                                      device=s["out"].device)
        for e, r0, r1 in experts:
            a = s["a"][tok[r0:r1]] if tok is not None else s["a"][r0:r1]
            dW[e] += s["dy"][r0:r1].double().t() @ a.double()
        return dW
    out = torch.empty(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    for e, r0, r1 in experts:
        if c["op"] == "dgrad":
            out[r0:r1] = s["dy"][r0:r1].double() @ s["W"][e].double()
            continue
        rows = s["x" if c["op"] == "q4" else "a"]
        rows = (rows[tok[r0:r1]] if tok is not None else rows[r0:r1]).double()
        if c["op"] == "gemm":
            out[r0:r1] = rows @ s["W"][e].double().t()
            continue
        slot = int(s["slot_of"][e])
        W = torch.empty(c["N"], c["K"], dtype=torch.float64, device=out.device)
        W[:, 0::2] = (s["codes"][slot] % 16).double()
        W[:, 1::2] = torch.div(s["codes"][slot], 16, rounding_mode="floor").double()
        if s["min"] is None:
            W -= 8
        W *= s["scale"][slot].double().repeat_interleave(c["group"], dim=1)
        if s["min"] is not None:
            W += s["min"][slot].double().repeat_interleave(c["group"], dim=1)
        y = rows @ W.t()
        if c["swiglu"]:
            half = c["N"] // 2
            y = y[:, :half] * torch.special.expit(y[:, :half]) * y[:, half:]
        out[r0:r1] = y
    return out
