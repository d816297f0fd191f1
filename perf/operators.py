"""Workloads of the quantised linear layer and of the mixture-of-experts layer.

Three operators, as a serving program calls them:

``scaled``   D = sA[i] * sB[j] * (A x B)(i, j) + bias[j], A and B int8 with one
             scale for each token (row of A) and channel (column of D); D bf16,
             fp16 or fp32 (``gemm_run_scaled``).
``linear``   the same layer on 16-bit activations: every token's row is quantised
             to int8 with its own scale (``gemm_quantize_rows``), then multiplied.
``moe``      a whole mixture-of-experts layer for a few tokens: softmax and top-k
             of the router's logits, the gate and up products of the chosen
             experts, silu(gate) * up, the down products and their weighted sum
             (``gemm_moe_run``); weights in the activations' 16-bit type, or int8
             with one scale for each output channel.

Weights are stored one output channel after the other, K contiguous, each line
padded to whole 16 bytes, as a program that loads them once would lay them out.
"""
import torch

own = False

F32, F16, BF16 = "f32", "f16", "bf16"
_TORCH = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}


def listed():
    return [
        # one decoded token through a square projection: latency
        {"name": "scaled_1x4096x4096_bf16", "op": "scaled", "M": 1, "N": 4096, "K": 4096,
         "out": BF16, "bias": False},
        # a decoding batch against the largest weights: the weights' bytes
        {"name": "scaled_16x16384x16384_f16", "op": "scaled", "M": 16, "N": 16384, "K": 16384,
         "out": F16, "bias": False},
        # a long prompt, or a training batch's forward: the matrix units
        {"name": "scaled_4096x4096x4096_bf16", "op": "scaled", "M": 4096, "N": 4096, "K": 4096,
         "out": BF16, "bias": False},
        # odd sizes with a bias and a 32-bit output (the last layer's logits)
        {"name": "scaled_3999x4001x4104_f32_bias", "op": "scaled", "M": 3999, "N": 4001,
         "K": 4104, "out": F32, "bias": True},
        # a small decoding batch on 16-bit activations: latency, two operators in a row
        {"name": "linear_8x4096x4096_bf16", "op": "linear", "M": 8, "N": 4096, "K": 4096,
         "out": BF16, "bias": True},
        # a larger decoding batch through a down projection
        {"name": "linear_64x4096x16384_bf16", "op": "linear", "M": 64, "N": 4096, "K": 16384,
         "out": BF16, "bias": False},
        # a prompt of 2048 tokens through an up projection
        {"name": "linear_2048x16384x4096_f16", "op": "linear", "M": 2048, "N": 16384, "K": 4096,
         "out": F16, "bias": True},
        # a small layer and one token, int8 weights: latency
        {"name": "moe_1_e8k2_1024x512_i8_bf16", "op": "moe", "T": 1, "H": 1024, "I": 512, "E": 8,
         "k": 2, "x": BF16, "i8": True, "renorm": True},
        # one token, many small experts
        {"name": "moe_1_e64k8_2048x1024_bf16", "op": "moe", "T": 1, "H": 2048, "I": 1024, "E": 64,
         "k": 8, "x": BF16, "i8": False, "renorm": False},
        # a decoding batch that reaches most experts
        {"name": "moe_16_e64k8_2048x1024_bf16", "op": "moe", "T": 16, "H": 2048, "I": 1024,
         "E": 64, "k": 8, "x": BF16, "i8": False, "renorm": True},
        # an odd batch and an inner width that ends inside a tile
        {"name": "moe_7_e16k4_4096x1000_f16", "op": "moe", "T": 7, "H": 4096, "I": 1000, "E": 16,
         "k": 4, "x": F16, "i8": False, "renorm": True},
        # the largest batch of the few-token layer, int8 weights
        {"name": "moe_64_e32k4_4096x2048_i8_bf16", "op": "moe", "T": 64, "H": 4096, "I": 2048,
         "E": 32, "k": 4, "x": BF16, "i8": True, "renorm": True},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi], odd ones among them."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.6:  # as most layers have it: a multiple of 64 where that is near
        n = max(lo, n // 64 * 64) if n >= 128 else n
    return min(hi, max(lo, n))


def draw(rng):
    if rng.random() < 0.55:
        op = rng.choice(["scaled", "linear"])
        while True:
            c = {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 256, 16384),
                 "K": _log(rng, 256, 16384), "out": rng.choice([BF16, F16, F32]),
                 "bias": rng.random() < 0.5}
            if c["M"] * c["N"] * c["K"] <= 1 << 36:
                return c
    while True:
        c = {"op": "moe", "T": _log(rng, 1, 64), "H": _log(rng, 512, 4096),
             "I": _log(rng, 256, 4096), "E": rng.choice([8, 16, 24, 32, 64, 128]),
             "k": rng.choice([1, 2, 4, 6, 8]), "x": rng.choice([BF16, F16]),
             "i8": rng.random() < 0.5, "renorm": rng.random() < 0.5}
        if c["E"] * c["I"] * c["H"] <= 1 << 28:
            return c


def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale


def _lines(values, per):
    """Rows whose stride is a multiple of `per` elements; the padding is part of no row."""
    rows, cols = values.shape
    ld = (cols + per - 1) // per * per
    store = torch.zeros(rows, ld, dtype=values.dtype, device=values.device)
    store[:, :cols] = values
    return store[:, :cols]


def _weights_i8(gen, rows, cols):
    """int8 weights of one scale for each channel: normal values, the largest of a channel 127."""
    q = (_normal(gen, rows, cols) * 32).round_().clamp_(-127, 127).to(torch.int8)
    scale = (torch.rand(rows, generator=gen, device="cuda") + 0.5) / (32 * cols ** 0.5)
    return _lines(q, 16), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "moe":
        T, H, I, E = case["T"], case["H"], case["I"], case["E"]
        x = _TORCH[case["x"]]
        s["X"] = _lines(_normal(gen, T, H).to(x), 8)
        # a trained router prefers some experts: its logits spread over a few units
        s["logits"] = _normal(gen, T, E, scale=1.5)
        if case["i8"]:
            s["W1"], s["s1"] = _weights_i8(gen, E * 2 * I, H)
            s["W2"], s["s2"] = _weights_i8(gen, E * H, I)
        else:
            s["W1"] = _lines(_normal(gen, E * 2 * I, H, scale=H ** -0.5).to(x), 8)
            s["W2"] = _lines(_normal(gen, E * H, I, scale=I ** -0.5).to(x), 8)
        s["D"] = torch.empty(T, H, dtype=x, device="cuda")
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["B"], s["sB"] = _weights_i8(gen, N, K)
    if case["bias"]:
        s["bias_values"] = _normal(gen, N, scale=0.1)
    # activations: normal, each token of another size, a few channels larger than the rest
    X = _normal(gen, M, K) * (0.25 + 2 * torch.rand(M, 1, generator=gen, device="cuda"))
    X[:, torch.randint(0, K, (max(1, K // 256),), generator=gen, device="cuda")] *= 6
    if case["op"] == "linear":
        s["X"] = _lines(X.to(torch.bfloat16 if case["out"] != F16 else torch.float16), 8)
        s["Q"] = torch.empty(M, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")
        s["sA"] = torch.empty(M, dtype=torch.float32, device="cuda")
    else:
        top = X.abs().amax(1, keepdim=True)
        s["A"] = _lines((X * (127 / top)).round().to(torch.int8), 16)
        s["sA"] = (top / 127).reshape(M)
    s["D"] = torch.empty(M, N, dtype=_TORCH[case["out"]], device="cuda")
    return s


def run(state):
    if own:
        return _framework(state)
    if state["op"] == "moe":
        return _plain_moe(state)
    if state["op"] == "linear":
        # round(x * 127 / max|x|) in 64 bits: a value next to a half must fall the right way
        x = state["X"].double()
        top = x.abs().amax(1, keepdim=True)
        q = torch.where(top > 0, x * 127 / top, 0.0).round().float()
        scale = (top / 127).float()
    else:
        q, scale = state["A"].float(), state["sA"].unsqueeze(1)
    d = torch.mm(q, state["B"].float().t()) * scale * state["sB"]
    if state["bias"]:
        d = d + state["bias_values"]
    return d.to(state["D"].dtype)


def _plain_moe(s):
    T, H, I, E, k = s["T"], s["H"], s["I"], s["E"], s["k"]
    e = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
    p, ids = torch.sort(e / e.sum(1, keepdim=True), dim=1, descending=True, stable=True)
    p, ids = p[:, :k], ids[:, :k]  # ties: the lowest expert first
    if s["renorm"]:
        p = p / p.sum(1, keepdim=True)
    w1, w2 = s["W1"].view(E, 2 * I, H), s["W2"].view(E, H, I)
    x = s["X"].float()
    if T * k < E:
        # few tokens: only the chosen experts' weights, one copy for each pair
        pair = ids.reshape(-1)
        w1, w2 = w1[pair].float(), w2[pair].float()
        if s["i8"]:
            w1 = w1 * s["s1"].view(E, 2 * I, 1)[pair]
            w2 = w2 * s["s2"].view(E, H, 1)[pair]
        up = torch.bmm(w1, x.repeat_interleave(k, 0).unsqueeze(2))
        h = up[:, :I] / (1 + torch.exp(-up[:, :I])) * up[:, I:]
        y = torch.bmm(w2, h).view(T, k, H)
        return (y * p.unsqueeze(2)).sum(1).to(s["D"].dtype)
    # more tokens than that: every expert on every token, weight 0 where it was not chosen
    w1, w2 = w1.float(), w2.float()
    if s["i8"]:
        w1, w2 = w1 * s["s1"].view(E, 2 * I, 1), w2 * s["s2"].view(E, H, 1)
    up = torch.mm(w1.reshape(E * 2 * I, H), x.t().contiguous()).view(E, 2 * I, T)
    h = up[:, :I] / (1 + torch.exp(-up[:, :I])) * up[:, I:]
    weight = torch.zeros(T, E, device="cuda").scatter(1, ids, p)
    y = torch.bmm(w2, h) * weight.t().unsqueeze(1)
    return y.sum(0).t().contiguous().to(s["D"].dtype)


def _framework(s):
    import dense_mixed_precision_tiled_amd as lg

    stream = torch.cuda.current_stream().cuda_stream
    types = {torch.float32: lg.GEMM_F32, torch.float16: lg.GEMM_F16, torch.bfloat16: lg.GEMM_BF16}
    D = s["D"]
    if s["op"] == "moe":
        if "layer" not in s:  # what a program makes once for each layer
            s["layer"] = lg.GemmMoe(
                H=s["H"], I=s["I"], E=s["E"], topk=s["k"],
                w_dtype=lg.GEMM_I8 if s["i8"] else types[D.dtype],
                W1=s["W1"].data_ptr(), ld1=s["W1"].stride(0),
                W2=s["W2"].data_ptr(), ld2=s["W2"].stride(0),
                scale1=s["s1"].data_ptr() if s["i8"] else 0,
                scale2=s["s2"].data_ptr() if s["i8"] else 0,
                activation=lg.GEMM_ACT_SILU, renormalize=s["renorm"])
            s["workspace"] = torch.empty(lg.gemm_moe_workspace(s["T"], s["layer"]),
                                         dtype=torch.uint8, device="cuda")
        X, logits, ws = s["X"], s["logits"], s["workspace"]
        st = lg.gemm_moe_run(s["T"], s["layer"], X.data_ptr(), X.stride(0), logits.data_ptr(),
                             logits.stride(0), D.data_ptr(), D.stride(0), types[X.dtype],
                             ws.data_ptr(), ws.numel(), stream)
        if st != lg.GEMM_OK:
            raise lg.GemmError(st, "gemm_moe_run")
        return D
    M, N, K, B = s["M"], s["N"], s["K"], s["B"]
    if s["op"] == "linear":
        X, A = s["X"], s["Q"]
        st = lg.gemm_quantize_rows(M, K, X.data_ptr(), X.stride(0), types[X.dtype], A.data_ptr(),
                                   A.stride(0), s["sA"].data_ptr(), stream)
        if st != lg.GEMM_OK:
            raise lg.GemmError(st, "gemm_quantize_rows")
    else:
        A = s["A"]
    if "epilogue" not in s:
        s["epilogue"] = lg.GemmEpilogue(bias=s["bias_values"].data_ptr()) if s["bias"] else None
    st = lg.gemm_run_scaled(M, N, K, A.data_ptr(), A.stride(0), lg.GEMM_ROW_MAJOR, B.data_ptr(),
                            B.stride(0), lg.GEMM_COL_MAJOR, s["sA"].data_ptr(),
                            s["sB"].data_ptr(), None, N, D.data_ptr(), D.stride(0), lg.GEMM_I8,
                            lg.GEMM_I32, types[D.dtype], 0, s["epilogue"], stream)
    if st != lg.GEMM_OK:
        raise lg.GemmError(st, "gemm_run_scaled")
    return D


def work(case):
    if case["op"] == "moe":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        k = min(k, E)
        # experts that T tokens of k reach, were the router even: the least that is read
        reached = max(k, round(E * (1 - (1 - k / E) ** T)))
        per = 3 * H * I * (1 if case["i8"] else 2) + (4 * (2 * I + H) if case["i8"] else 0)
        return {"bytes": reached * per + 4 * T * H + 4 * T * E, "flops": 6 * T * k * H * I}
    M, N, K = case["M"], case["N"], case["K"]
    size = 4 if case["out"] == F32 else 2
    a = M * K * (2 if case["op"] == "linear" else 1) + (0 if case["op"] == "linear" else 4 * M)
    return {"bytes": a + N * K + 4 * N + (4 * N if case["bias"] else 0) + M * N * size,
            "flops": 2 * M * N * K}


def exact(case, seed):
    """From the definitions in 64 bits, one channel block or expert at a time."""
    s = prepare(case, seed)
    if case["op"] != "moe":
        if case["op"] == "linear":
            x = s["X"].to(torch.float64)
            largest = x.abs().max(dim=1).values
            # 127 x is exact, so a tie stays one
            a = torch.round(127 * x / torch.where(largest > 0, largest, 1.0)[:, None])
            step = largest / 127
        else:
            a, step = s["A"].to(torch.float64), s["sA"].to(torch.float64)
        out = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for j in range(0, case["N"], 4096):
            out[:, j:j + 4096] = a @ s["B"][j:j + 4096].to(torch.float64).t()
        out *= step[:, None]
        out *= s["sB"].to(torch.float64)
        return out + s["bias_values"].to(torch.float64) if case["bias"] else out
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    prob = torch.softmax(s["logits"].to(torch.float64), dim=1).cpu()
    keys = s["logits"].cpu().tolist()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    chosen = [sorted(range(E), key=lambda e: (-row[e], e))[:k] for row in keys]
    for e in range(E):
        rows = [t for t in range(T) if e in chosen[t]]
        if not rows:
            continue
        w1 = s["W1"][e * 2 * I:(e + 1) * 2 * I].to(torch.float64)
        w2 = s["W2"][e * H:(e + 1) * H].to(torch.float64)
        if case["i8"]:
            w1 = w1 * s["s1"][e * 2 * I:(e + 1) * 2 * I].to(torch.float64)[:, None]
            w2 = w2 * s["s2"][e * H:(e + 1) * H].to(torch.float64)[:, None]
        x = s["X"][rows].to(torch.float64)
        gate, up = x @ w1[:I].t(), x @ w1[I:].t()
        y = (gate * torch.sigmoid(gate) * up) @ w2.t()
        share = [float(prob[t, e]) / (float(prob[t, chosen[t]].sum()) if case["renorm"] else 1.0)
                 for t in rows]
        out[rows] += y * torch.tensor(share, dtype=torch.float64, device="cuda")[:, None]
    return out
