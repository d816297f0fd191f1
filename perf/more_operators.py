"""Workloads of adapters, 8-bit activation checkpoints and the router's balance loss.

Four operators, as a training or serving program calls them:

``adapters``    low-rank adapters of many requests at once beside a shared projection:
                D(t) = C(t) + scale[a] * (x_t A_a^T) B_a^T with a = ids[t], and D(t) =
                C(t) for a token without one (``gemm_lora_run``).  C is the shared
                projection's output.
``checkpoint``  activations kept in 8 bits for the backward pass: packed
                (``gemm_checkpoint_pack``), then taken back, as values
                (``gemm_checkpoint_unpack``) or as the gradient of an activation
                function on them, D = G * act'(X) (``gemm_checkpoint_act_grad``).
``wgrad``       a linear layer's weight gradient from packed activations, added to
                the gradient so far: D = G^T X + C (``gemm_checkpoint_wgrad``).
``balance``     a router's balance loss and per-expert counts, forward and backward
                (``gemm_moe_balance``, ``gemm_moe_balance_grad``).

Packed activations: 32 consecutive values of a row share a power of two, stored as
one byte S; the values are int8, X = 2^(S - 127) * Q / 64.
"""
import torch

own = False

F32, F16, BF16 = "f32", "f16", "bf16"
_TORCH = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}


def listed():
    return [
        # one decoded token with its adapter: latency
        {"name": "adapters_1x4096x4096_r16_bf16", "op": "adapters", "T": 1, "K": 4096, "N": 4096,
         "rank": 16, "adapters": 16, "none": False, "segments": 0, "x": BF16, "out": BF16},
        # a decoding batch in which every request has another adapter
        {"name": "adapters_64x4096x4096_r16_bf16", "op": "adapters", "T": 64, "K": 4096, "N": 4096,
         "rank": 16, "adapters": 64, "none": False, "segments": 0, "x": BF16, "out": BF16},
        # an odd batch, some requests without an adapter; ragged widths and rank, fp32 logits
        {"name": "adapters_37x4104x4001_r12_f16_f32", "op": "adapters", "T": 37, "K": 4104,
         "N": 4001, "rank": 12, "adapters": 9, "none": True, "segments": 0, "x": F16, "out": F32},
        # packed prompts of different requests
        {"name": "adapters_4096x4096x4096_r64_bf16", "op": "adapters", "T": 4096, "K": 4096,
         "N": 4096, "rank": 64, "adapters": 8, "none": True, "segments": 12, "x": BF16,
         "out": BF16},
        # a small micro-batch's activations, a width that ends inside a block of 32
        {"name": "checkpoint_100x4104_f16", "op": "checkpoint", "M": 100, "K": 4104, "x": F16,
         "act": "none"},
        # an inner layer's values before its activation function, a whole training batch
        {"name": "checkpoint_4096x16384_gelu_bf16", "op": "checkpoint", "M": 4096, "K": 16384,
         "x": BF16, "act": "gelu"},
        # a router's, or an adapter's first matrix's, gradient: few outputs, many tokens
        {"name": "wgrad_16x4096_of_8192_bf16_f32", "op": "wgrad", "M": 8192, "N": 16, "K": 4096,
         "x": BF16, "out": F32, "add": False},
        # an odd layer and batch with loss-scaled fp16 gradients
        {"name": "wgrad_1001x2056_of_3999_f16", "op": "wgrad", "M": 3999, "N": 1001, "K": 2056,
         "x": F16, "out": F16, "add": False},
        # a square projection, added to the fp32 gradient of earlier micro-batches
        {"name": "wgrad_4096x4096_of_4096_bf16_f32", "op": "wgrad", "M": 4096, "N": 4096, "K": 4096,
         "x": BF16, "out": F32, "add": True},
        # a small router on one short batch: latency, four calls' launches
        {"name": "balance_1024x8_k2", "op": "balance", "T": 1024, "E": 8, "k": 2, "mask": False,
         "out": F32},
        # a padded batch, an odd number of experts
        {"name": "balance_8191x60_k4_mask", "op": "balance", "T": 8191, "E": 60, "k": 4,
         "mask": True, "out": F32},
        # many small experts, a whole training batch; 16-bit gradients for the products behind
        {"name": "balance_65536x64_k8_bf16", "op": "balance", "T": 65536, "E": 64, "k": 8,
         "mask": False, "out": BF16},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi], odd ones among them."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 0.5:  # as most layers have it: a multiple of 64 where that is near
        n = max(lo, n // 64 * 64) if n >= 128 else n
    return min(hi, max(lo, n))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "checkpoint", "wgrad", "wgrad", "balance"])
    if op == "adapters":
        while True:
            c = {"op": op, "T": _log(rng, 1, 4096), "K": _log(rng, 256, 8192),
                 "N": _log(rng, 256, 8192), "rank": rng.choice([4, 8, 12, 16, 24, 32, 64]),
                 "adapters": _log(rng, 1, 64), "none": rng.random() < 0.5, "segments": 0,
                 "x": rng.choice([BF16, F16])}
            c["out"] = rng.choice([c["x"], c["x"], F32])
            if c["T"] > 256:
                c["segments"] = rng.randint(1, 24)
            if c["T"] * (c["K"] + c["N"]) <= 1 << 25 and c["adapters"] * c["rank"] <= 512:
                return c
    if op == "checkpoint":
        while True:
            c = {"op": op, "M": _log(rng, 1, 16384), "K": _log(rng, 64, 16384),
                 "x": rng.choice([BF16, BF16, F16]),
                 "act": rng.choice(["none", "relu", "gelu", "silu"])}
            if c["M"] * c["K"] <= 1 << 26:
                return c
    if op == "wgrad":
        while True:
            c = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 8, 8192),
                 "K": _log(rng, 64, 8192), "x": rng.choice([BF16, BF16, F16]),
                 "add": rng.random() < 0.5}
            c["out"] = rng.choice([c["x"], F32])
            if c["M"] * c["N"] * c["K"] <= 1 << 36 and c["M"] * (c["N"] + c["K"]) <= 1 << 26:
                return c
    while True:
        c = {"op": op, "T": _log(rng, 1, 65536), "E": _log(rng, 4, 256), "mask": rng.random() < 0.5,
             "out": rng.choice([F32, BF16])}
        c["k"] = min(c["E"], rng.choice([1, 2, 4, 6, 8]))
        if c["T"] * c["E"] <= 1 << 22:
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


def _activations(gen, M, K):
    """Normal values, each token of another size, a few channels larger than the rest."""
    X = _normal(gen, M, K) * (0.25 + 2 * torch.rand(M, 1, generator=gen, device="cuda"))
    X[:, torch.randint(0, K, (max(1, K // 256),), generator=gen, device="cuda")] *= 6
    return X


def _pack(X):
    """(Q, S) of the packed format, from the definition."""
    M, K = X.shape
    blocks = (K + 31) // 32
    x = torch.zeros(M, blocks * 32, dtype=torch.float64, device=X.device)
    x[:, :K] = X
    x = x.view(M, blocks, 32)
    top = x.abs().amax(2)
    e = torch.frexp(top).exponent - 1  # floor(log2(top))
    s = torch.where(top > 0, (e + 127).clamp(0, 254), 0)
    q = torch.round(torch.ldexp(x, (133 - s).unsqueeze(2))).clamp(-127, 127)
    return q.view(M, -1)[:, :K].to(torch.int8), s.to(torch.uint8)


def _values(Q, S, dtype):
    """What packed activations stand for."""
    M, K = Q.shape
    step = torch.ldexp(torch.ones((), dtype=torch.float64, device=Q.device), S.to(torch.int32) - 133)
    return Q.to(dtype) * step.to(dtype).repeat_interleave(32, 1)[:, :K]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] == "adapters":
        T, K, N, r, n = (case[f] for f in ("T", "K", "N", "rank", "adapters"))
        x, out = _TORCH[case["x"]], _TORCH[case["out"]]
        s["X"] = _lines(_activations(gen, T, K).to(x), 8)
        s["A"] = _lines(_normal(gen, n * r, K, scale=K ** -0.5).to(x), 8)
        s["B"] = _lines(_normal(gen, n * N, r, scale=r ** -0.5).to(x), 8)
        s["scales"] = 0.5 + torch.rand(n, generator=gen, device="cuda")
        s["C"] = _lines(_normal(gen, T, N).to(out), 8)
        s["D"] = _lines(torch.empty(T, N, dtype=out, device="cuda"), 8)
        # a request for each token, or packed prompts of several requests
        if case["segments"]:
            cuts = torch.randint(0, T, (case["segments"] - 1,), generator=gen, device="cuda")
            ends = torch.sort(cuts).values
            request = torch.searchsorted(ends, torch.arange(T, device="cuda"), right=True)
        else:
            request = torch.randperm(T, generator=gen, device="cuda")
        ids = request % n
        if case["none"]:  # every fifth request uses the shared projection alone
            ids = torch.where(request % 5 == 4, -1, ids)
        s["ids"] = ids.to(torch.int32)
    elif case["op"] == "checkpoint":
        M, K, x = case["M"], case["K"], _TORCH[case["x"]]
        s["X"] = _lines(_activations(gen, M, K).to(x), 8)
        s["Q"] = _lines(torch.zeros(M, K, dtype=torch.int8, device="cuda"), 16)
        s["S"] = torch.zeros(M, (K + 31) // 32, dtype=torch.uint8, device="cuda")
        s["D"] = _lines(torch.empty(M, K, dtype=x, device="cuda"), 8)
        if case["act"] != "none":
            s["G"] = _lines(_normal(gen, M, K).to(x), 8)
    elif case["op"] == "wgrad":
        M, N, K, x, out = case["M"], case["N"], case["K"], _TORCH[case["x"]], _TORCH[case["out"]]
        Q, s["S"] = _pack(_activations(gen, M, K).to(x))
        s["Q"] = _lines(Q, 16)
        s["G"] = _lines(_normal(gen, M, N, scale=M ** -0.5).to(x), 8)
        s["C"] = _normal(gen, N, K).to(out) if case["add"] else None
        s["D"] = torch.empty(N, K, dtype=out, device="cuda")
    else:
        T, E = case["T"], case["E"]
        # a trained router prefers some experts: its logits spread over a few units
        s["logits"] = _normal(gen, T, E, scale=1.5) + _normal(gen, 1, E, scale=0.5)
        s["mask"] = None
        if case["mask"]:  # about a tenth of the batch is padding
            s["mask"] = (torch.rand(T, generator=gen, device="cuda") < 0.9).to(torch.uint8)
            s["mask"][0] = 1
        s["dloss"] = 0.5 + torch.rand(1, generator=gen, device="cuda")
        s["loss"] = torch.empty(3, device="cuda")
        s["counts"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        s["lse"] = torch.empty(T, device="cuda")
        s["D"] = torch.empty(T, E, dtype=_TORCH[case["out"]], device="cuda")
    return s


BALANCE, Z = 0.01, 0.001  # the two terms' usual weights


def run(state):
    if own:
        return _framework(state)
    return {"adapters": _plain_adapters, "checkpoint": _plain_checkpoint, "wgrad": _plain_wgrad,
            "balance": _plain_balance}[state["op"]](state)


def _plain_adapters(s):
    T, K, N, r, n = (s[f] for f in ("T", "K", "N", "rank", "adapters"))
    x, ids = s["X"].float(), s["ids"].long()
    has = ids >= 0
    a = ids.clamp(min=0)
    A, B = s["A"].reshape(n, r, K), s["B"].reshape(n, N, r)
    if T <= 2 * n:
        # few tokens: each token's own weights
        h = torch.bmm(A[a].float(), x.unsqueeze(2))
        y = torch.bmm(B[a].float(), h).squeeze(2)
    else:
        # more: every adapter on every token, then each token's own
        h = torch.mm(x, A.float().view(n * r, K).t()).view(T, n, r)
        own_h = torch.zeros(T, n, r, device="cuda")
        rows = torch.arange(T, device="cuda")
        own_h[rows, a] = h[rows, a]
        y = torch.mm(own_h.view(T, n * r), B.float().transpose(1, 2).reshape(n * r, N))
    y = torch.where(has.unsqueeze(1), y * s["scales"][a].unsqueeze(1), 0.0)
    return (s["C"].float() + y).to(s["D"].dtype)


def _slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu":
        phi = torch.exp(-0.5 * x * x) * 0.3989422804014327
        return 0.5 * torch.erfc(x * -0.7071067811865476) + x * phi
    sig = 1 / (1 + torch.exp(-x))
    return sig * (1 + x * (1 - sig))


def _plain_checkpoint(s):
    X = s["X"]
    M, K = X.shape
    blocks = (K + 31) // 32
    x = torch.zeros(M, blocks * 32, device="cuda")
    x[:, :K] = X
    x = x.view(M, blocks, 32)
    top = x.abs().amax(2)
    e = torch.where(top > 0, torch.frexp(top).exponent - 1, -127).clamp(min=-127).unsqueeze(2)
    q = torch.round(torch.ldexp(x, 6 - e)).clamp(-127, 127).to(torch.int8)
    y = torch.ldexp(q.float(), e - 6).view(M, -1)[:, :K]
    if s["act"] != "none":
        y = s["G"].float() * _slope(y, s["act"])
    return y.to(X.dtype)


def _plain_wgrad(s):
    d = torch.mm(s["G"].float().t(), _values(s["Q"], s["S"], torch.float32))
    if s["C"] is not None:
        d = d + s["C"].float()
    return d.to(s["D"].dtype)


def _plain_balance(s):
    T, E, k = s["T"], s["E"], s["k"]
    logits = s["logits"]
    live = torch.ones(T, device="cuda") if s["mask"] is None else (s["mask"] != 0).float()
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    p, lse = e / total * live.unsqueeze(1), (torch.log(total) + top).squeeze(1) * live
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = torch.zeros(T, E, device="cuda").scatter(1, order, 1.0) * live.unsqueeze(1)
    n = live.double().sum()  # sums over tokens in 64 bits
    counts = chosen.double().sum(0)
    f, mean = counts / (n * k), p.double().sum(0) / n
    terms = torch.stack([E * (f * mean).sum(), (lse.double() ** 2).sum() / n])
    loss = torch.cat([(BALANCE * terms[0] + Z * terms[1]).view(1), terms]).float()
    f, g = f.float(), s["dloss"] / n.float()
    pull = BALANCE * E * (f - (p * f).sum(1, keepdim=True)) + 2 * Z * lse.unsqueeze(1)
    return {"loss": loss, "counts": torch.cat([counts, n.view(1)]).to(torch.int32), "lse": lse,
            "dlogits": (g * p * pull).to(s["D"].dtype)}


def _check(lg, status, name):
    if status != lg.GEMM_OK:
        raise lg.GemmError(status, name)


def _workspace(s, size):
    """The call's workspace, kept beside the plan as a program keeps it."""
    if size < 0:
        raise ValueError("workspace: status %d" % size)
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(1, size), dtype=torch.uint8, device="cuda")
    return s["workspace"].data_ptr(), s["workspace"].numel()


def _framework(s):
    import dense_mixed_precision_tiled_amd as lg

    stream = torch.cuda.current_stream().cuda_stream
    types = {torch.float32: lg.GEMM_F32, torch.float16: lg.GEMM_F16, torch.bfloat16: lg.GEMM_BF16}
    D = s["D"]
    if s["op"] == "adapters":
        if "lora" not in s:  # what a program makes once for each projection
            s["lora"] = lg.GemmLora(K=s["K"], N=s["N"], adapters=s["adapters"], rank=s["rank"],
                                    A=s["A"].data_ptr(), lda=s["A"].stride(0),
                                    B=s["B"].data_ptr(), ldb=s["B"].stride(0),
                                    scales=s["scales"].data_ptr())
        X, C = s["X"], s["C"]
        ws, size = _workspace(s, lg.gemm_lora_workspace(s["T"], s["lora"]))
        _check(lg, lg.gemm_lora_run(s["T"], s["lora"], X.data_ptr(), X.stride(0),
                                    s["ids"].data_ptr(), C.data_ptr(), C.stride(0), D.data_ptr(),
                                    D.stride(0), types[X.dtype], types[D.dtype], ws, size, stream),
               "gemm_lora_run")
        return D
    if s["op"] == "checkpoint":
        M, K, X, Q, S = s["M"], s["K"], s["X"], s["Q"], s["S"]
        _check(lg, lg.gemm_checkpoint_pack(M, K, X.data_ptr(), X.stride(0), types[X.dtype],
                                           Q.data_ptr(), Q.stride(0), S.data_ptr(), S.stride(0),
                                           stream), "gemm_checkpoint_pack")
        if s["act"] == "none":
            _check(lg, lg.gemm_checkpoint_unpack(M, K, Q.data_ptr(), Q.stride(0), S.data_ptr(),
                                                 S.stride(0), D.data_ptr(), D.stride(0),
                                                 types[D.dtype], stream), "gemm_checkpoint_unpack")
            return D
        act = {"relu": lg.GEMM_ACT_RELU, "gelu": lg.GEMM_ACT_GELU, "silu": lg.GEMM_ACT_SILU}
        G = s["G"]
        _check(lg, lg.gemm_checkpoint_act_grad(M, K, Q.data_ptr(), Q.stride(0), S.data_ptr(),
                                               S.stride(0), G.data_ptr(), G.stride(0),
                                               act[s["act"]], D.data_ptr(), D.stride(0),
                                               types[D.dtype], stream), "gemm_checkpoint_act_grad")
        return D
    if s["op"] == "wgrad":
        M, N, K, G, Q, S, C = (s[f] for f in ("M", "N", "K", "G", "Q", "S", "C"))
        ws, size = _workspace(s, lg.gemm_checkpoint_wgrad_workspace(M, N, K))
        _check(lg, lg.gemm_checkpoint_wgrad(M, N, K, G.data_ptr(), G.stride(0), Q.data_ptr(),
                                            Q.stride(0), S.data_ptr(), S.stride(0),
                                            0 if C is None else C.data_ptr(), K, D.data_ptr(), K,
                                            types[G.dtype], types[D.dtype], ws, size, stream),
               "gemm_checkpoint_wgrad")
        return D
    T, E, k, logits = s["T"], s["E"], s["k"], s["logits"]
    mask = 0 if s["mask"] is None else s["mask"].data_ptr()
    loss, counts, lse = s["loss"], s["counts"], s["lse"]
    ws, size = _workspace(s, lg.gemm_moe_balance_workspace(T, E, k))
    _check(lg, lg.gemm_moe_balance(T, E, k, logits.data_ptr(), logits.stride(0), mask, BALANCE, Z,
                                   loss.data_ptr(), counts.data_ptr(), lse.data_ptr(), ws, size,
                                   stream), "gemm_moe_balance")
    _check(lg, lg.gemm_moe_balance_grad(T, E, k, logits.data_ptr(), logits.stride(0), mask, BALANCE,
                                        Z, counts.data_ptr(), lse.data_ptr(),
                                        s["dloss"].data_ptr(), D.data_ptr(), D.stride(0),
                                        types[D.dtype], stream), "gemm_moe_balance_grad")
    return {"loss": loss, "counts": counts, "lse": lse, "dlogits": D}


def _size(dtype):
    return 4 if dtype == F32 else 2


def work(case):
    if case["op"] == "adapters":
        T, K, N, r = (case[f] for f in ("T", "K", "N", "rank"))
        requests = case["segments"] or T
        reached = min(case["adapters"], requests)
        with_one = T * 0.8 if case["none"] else T
        return {"bytes": 2 * T * K + 2 * T * N * _size(case["out"]) + 4 * T +
                reached * (2 * r * (K + N) + 4),
                "flops": 2 * int(with_one) * r * (K + N)}
    if case["op"] == "checkpoint":
        values = case["M"] * case["K"]
        packed = values + case["M"] * ((case["K"] + 31) // 32)
        # forward: values in, packed out; backward: packed (and a gradient) in, values out
        return {"bytes": 2 * values + 2 * packed + (4 if case["act"] != "none" else 2) * values,
                "flops": (4 if case["act"] == "none" else 24) * values}
    if case["op"] == "wgrad":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * N + M * (K + (K + 31) // 32) +
                (2 if case["add"] else 1) * N * K * _size(case["out"]),
                "flops": 2 * M * N * K}
    T, E = case["T"], case["E"]
    # forward: logits in, lse out; backward: logits and lse in, gradients out
    return {"bytes": 8 * T * E + 8 * T + (2 * T if case["mask"] else 0) + T * E * _size(case["out"]),
            "flops": 30 * T * E}


def exact(case, seed):
    """From the definitions in 64 bits, one adapter, row block or token block at a time."""
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "adapters":
        K, N, r = case["K"], case["N"], case["rank"]
        out = s["C"].to(f64)
        for i in range(case["adapters"]):
            rows = torch.nonzero(s["ids"] == i).squeeze(1)
            if rows.numel() == 0:
                continue
            down = s["A"][i * r:(i + 1) * r].to(f64)
            up = s["B"][i * N:(i + 1) * N].to(f64)
            out[rows] += float(s["scales"][i]) * ((s["X"][rows].to(f64) @ down.t()) @ up.t())
        return out
    if case["op"] == "checkpoint":
        out = torch.empty(case["M"], case["K"], dtype=f64, device="cuda")
        for i in range(0, case["M"], 1024):
            block = slice(i, i + 1024)
            x = _values(*_pack(s["X"][block]), f64)
            if case["act"] == "gelu":
                cdf = torch.special.ndtr(x)
                x = s["G"][block].to(f64) * (cdf + x * torch.exp(-x * x / 2) / (2 * torch.pi) ** 0.5)
            elif case["act"] == "silu":
                gate = torch.sigmoid(x)
                x = s["G"][block].to(f64) * (gate + x * gate * (1 - gate))
            elif case["act"] == "relu":
                x = torch.where(x > 0, s["G"][block].to(f64), 0.0)
            out[block] = x
        return out
    if case["op"] == "wgrad":
        out = torch.zeros(case["N"], case["K"], dtype=f64, device="cuda")
        if s["C"] is not None:
            out += s["C"].to(f64)
        for i in range(0, case["M"], 2048):
            x = _values(s["Q"][i:i + 2048], s["S"][i:i + 2048], f64)
            out += s["G"][i:i + 2048].to(f64).t() @ x
        return out
    T, E, k = case["T"], case["E"], case["k"]
    logits = s["logits"].to(f64)
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    lse = torch.where(live, torch.logsumexp(logits, 1), 0.0)
    p = torch.where(live[:, None], torch.softmax(logits, 1), 0.0)
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    counts[E] = live.sum()
    left = s["logits"].clone()
    for _ in range(k):  # the largest one left, the first of equal ones
        top = left.max(1, keepdim=True).values
        first = torch.argmax((left == top).to(torch.int32), 1)
        counts[:E] += torch.bincount(first[live], minlength=E)
        left.scatter_(1, first[:, None], float("-inf"))
    n = float(counts[E])
    share = counts[:E].to(f64) / (n * k)
    balance = E * (share @ p.sum(0)) / n
    z = (lse * lse).sum() / n
    dp = BALANCE * E * share
    inner = p @ dp
    d = p * (dp[None, :] - inner[:, None]) + 2 * Z * (lse[:, None] * p)
    return {"loss": torch.stack([BALANCE * balance + Z * z, balance, z]),
            "counts": counts.to(torch.int32), "lse": lse, "dlogits": d * (float(s["dloss"]) / n)}
