"""The 8-bit-float (e4m3) operators of a decoder layer: cases, inputs, plain forms and exact values.

norm     RMSNorm of x + residual, quantized to e4m3 with a scale per 128 channels of a row
quant    the quantizers: activations (per 128 of a row, SiLU-gated or not), weights (per 128 x 128)
gemm     Y = X·Wᵀ on e4m3 operands with those scales
grouped  the same product with an expert's weight per range of rows

`own` selects the package's entry points instead of the plain forms.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a 4096-wide layer: the norm in front of a decode step
        {"name": "norm_token", "op": "norm", "rows": 1, "dim": 4096, "dtype": "bf16",
         "residual": True, "want_y": False},
        # float32 activations, an odd batch and a width that ends inside a block
        {"name": "norm_odd_f32", "op": "norm", "rows": 777, "dim": 1040, "dtype": "f32",
         "residual": False, "want_y": True},
        # a prefill batch of an 8192-wide layer (one tuning minibatch of tokens)
        {"name": "norm_prefill", "op": "norm", "rows": 16384, "dim": 8192, "dtype": "bf16",
         "residual": True, "want_y": False},
        # the input of down_proj: SiLU(gate)·up of 2048 tokens, quantized
        {"name": "quant_gated", "op": "quant_act", "rows": 2048, "dim": 11008, "dtype": "bf16",
         "gate": True},
        # a 29568 x 8192 up_proj weight, quantized once when a layer is deployed
        {"name": "quant_weight", "op": "quant_weight", "experts": 1, "rows": 29568, "dim": 8192,
         "dtype": "bf16"},
        # decode of one token through q_proj
        {"name": "gemm_token", "op": "gemm", "rows": 1, "cols": 4096, "dim": 4096, "out": "bf16"},
        # decode of a batch of 16 through the largest Linear
        {"name": "gemm_decode_16", "op": "gemm", "rows": 16, "cols": 29568, "dim": 8192,
         "out": "bf16"},
        # a short odd prompt, float32 output, widths that end inside a block
        {"name": "gemm_odd_f32", "op": "gemm", "rows": 333, "cols": 2050, "dim": 1360,
         "out": "f32"},
        # prefill of one tuning minibatch through q_proj
        {"name": "gemm_prefill", "op": "gemm", "rows": 16384, "cols": 4096, "dim": 4096,
         "out": "bf16"},
        # decode of 24 tokens, 4 of 64 small experts each: most experts have a row or two
        {"name": "grouped_decode", "op": "grouped", "experts": 64, "tokens": 24, "topk": 4,
         "cols": 2048, "dim": 2048, "gather": True, "out": "bf16"},
        # an odd batch over a few experts whose widths end inside a block
        {"name": "grouped_odd", "op": "grouped", "experts": 9, "tokens": 701, "topk": 2,
         "cols": 1000, "dim": 720, "gather": False, "out": "f32"},
        # prefill of 8192 tokens, 2 of 8 experts of gate_proj's size each
        {"name": "grouped_prefill", "op": "grouped", "experts": 8, "tokens": 8192, "topk": 2,
         "cols": 11008, "dim": 4096, "gather": True, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant_act", "quant_weight", "gemm", "gemm", "grouped", "grouped"])
    if op == "norm":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "dim": 16 * _log_int(rng, 4, 512),
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "residual": rng.random() < 0.7,
                "want_y": rng.random() < 0.3}
    if op == "quant_act":
        gate = rng.random() < 0.6
        return {"op": op, "rows": _log_int(rng, 1, 8192 if gate else 16384),
                "dim": 16 * _log_int(rng, 4, 688), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "gate": gate}
    while True:
        if op == "quant_weight":
            c = {"op": op, "experts": _log_int(rng, 1, 16), "rows": _log_int(rng, 1, 29568),
                 "dim": 16 * _log_int(rng, 1, 688), "dtype": rng.choice(["bf16", "f32"])}
            if c["experts"] * c["rows"] * c["dim"] <= 29568 * 8192:
                return c
        elif op == "gemm":
            c = {"op": op, "rows": _log_int(rng, 1, 16384), "cols": _log_int(rng, 16, 29568),
                 "dim": 16 * _log_int(rng, 8, 688), "out": rng.choice(["bf16", "bf16", "f32"])}
            if c["rows"] * c["cols"] * c["dim"] <= 16384 * 4096 * 4096 and \
                    c["cols"] * c["dim"] <= 29568 * 8192:
                return c
        else:
            c = {"op": op, "experts": _log_int(rng, 2, 128), "tokens": _log_int(rng, 1, 8192),
                 "topk": rng.randint(1, 8), "cols": _log_int(rng, 64, 11008),
                 "dim": 16 * _log_int(rng, 8, 256), "gather": rng.random() < 0.5,
                 "out": rng.choice(["bf16", "bf16", "f32"])}
            if c["topk"] <= c["experts"] and c["tokens"] * c["topk"] <= 16384 and \
                    c["experts"] * c["cols"] * c["dim"] <= 8 * 11008 * 4096 and \
                    c["tokens"] * c["topk"] * c["cols"] * c["dim"] <= 16384 * 11008 * 4096:
                return c


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, dim, dtype):
    """N(0, 1) tokens in which one channel of a hundred is 20 times as large."""
    x = torch.randn((rows, dim), generator=g, device="cuda")
    big = torch.rand((dim,), generator=g, device="cuda") < 0.01
    return torch.where(big, 20.0 * x, x).to(dtype)


def _codes(x, amax, of):
    """e4m3 codes of x under the scales of the block maxima amax (spread over x by `of`)."""
    scale = torch.where(amax == 0, torch.ones_like(amax), (amax / E4M3_MAX).clamp(min=TINY))
    return (x / of(scale)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def _blocks(n):
    return -(-n // BLOCK)


def _quant_rows(x):
    """x [M, K] -> codes [M, K], scales [KB, M]: one per 128 channels of a row."""
    M, K = x.shape
    KB = _blocks(K)
    xp = torch.nn.functional.pad(x, (0, KB * BLOCK - K)).view(M, KB, BLOCK)
    q, s = _codes(xp, xp.abs().amax(-1, keepdim=True), lambda s: s)
    return q.view(M, KB * BLOCK)[:, :K].contiguous(), s.view(M, KB).t().contiguous()


def _quant_weight(w):
    """w [E, N, K] -> codes [E, N, K], scales [E, NB, KB]: one per 128 x 128 block."""
    E, N, K = w.shape
    NB, KB = _blocks(N), _blocks(K)
    wp = torch.nn.functional.pad(w, (0, KB * BLOCK - K, 0, NB * BLOCK - N))
    wp = wp.view(E, NB, BLOCK, KB, BLOCK)
    q, s = _codes(wp, wp.abs().amax((2, 4), keepdim=True), lambda s: s)
    q = q.view(E, NB * BLOCK, KB * BLOCK)[:, :N, :K].contiguous()
    return q, s.view(E, NB, KB)


def _weights(g, experts, rows, dim):
    """Codes and scales of N(0, 0.02) weights whose output rows differ in size."""
    q = torch.empty((experts, rows, dim), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((experts, _blocks(rows), _blocks(dim)), device="cuda")
    for e in range(experts):
        w = 0.02 * torch.randn((rows, dim), generator=g, device="cuda")
        w *= torch.rand((rows, 1), generator=g, device="cuda") + 0.5
        q[e:e + 1], s[e:e + 1] = _quant_weight(w[None])
    return q, s


def _routing(g, case):
    """Rows sorted by expert: offsets [E + 1], the token of each row, and the largest group.
    Every token picks topk different experts, some of them more popular than others."""
    E, T, k = case["experts"], case["tokens"], case["topk"]
    popular = 1.5 * torch.randn((E,), generator=g, device="cuda")
    u = torch.rand((T, E), generator=g, device="cuda").clamp(1e-9, 1 - 1e-7)
    chosen = (popular - torch.log(-torch.log(u))).topk(k, dim=1).indices.reshape(-1)
    order = torch.sort(chosen, stable=True).indices
    counts = torch.bincount(chosen, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    return offsets, (order // k).to(torch.int32), int(counts.max())


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "norm":
        dt = DTYPES[case["dtype"]]
        s["x"] = _activations(g, case["rows"], case["dim"], dt)
        s["residual"] = _activations(g, case["rows"], case["dim"], dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * torch.randn((case["dim"],), generator=g, device="cuda")).to(dt)
    elif op == "quant_act":
        dim = case["dim"] * (2 if case["gate"] else 1)
        s["x"] = _activations(g, case["rows"], dim, DTYPES[case["dtype"]])
    elif op == "quant_weight":
        shape = (case["experts"], case["rows"], case["dim"])
        s["w"] = (0.02 * torch.randn(shape, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    else:
        experts = case["experts"] if op == "grouped" else 1
        wq, ws = _weights(g, experts, case["cols"], case["dim"])
        if op == "grouped":
            s["offsets"], row, s["largest"] = _routing(g, case)
            rows = case["tokens"] if case["gather"] else case["tokens"] * case["topk"]
            s["row_index"] = row if case["gather"] else None
            s["wq"], s["ws"] = wq, ws
        else:
            rows = case["rows"]
            s["wq"], s["ws"] = wq[0], ws[0]
        s["xq"], s["xs"] = _quant_rows(_activations(g, rows, case["dim"], torch.float32))
    return s


# ------------------------------------------------------------------ plain forms
def _spread(s, dim, n):
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _norm(x, residual, weight, eps):
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    v = h.float()
    y = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * weight.float()
    return h, y


def _gated(x):
    a, b = x.float().chunk(2, dim=-1)
    return a / (1 + torch.exp(-a)) * b


def _product(xq, xs, wq, ws, out):
    x = xq.float() * _spread(xs, 0, xq.shape[1]).t()
    w = wq.float() * _spread(_spread(ws, 0, wq.shape[0]), 1, wq.shape[1])
    return (x @ w.t()).to(out)


def _grouped_product(xq, xs, wq, ws, offsets, row_index, largest, out):
    """Each expert's rows padded to the largest group's, one batched product."""
    E, N, K = wq.shape
    x = xq.float() * _spread(xs, 0, K).t()
    R = x.shape[0] if row_index is None else row_index.shape[0]
    row = torch.arange(R, dtype=torch.int32, device=x.device)
    e = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    place = e * largest + (row - offsets[e])
    padded = torch.zeros((E * largest, K), device=x.device)
    padded[place] = x if row_index is None else x[row_index.long()]
    w = wq.float() * _spread(_spread(ws, 1, N), 2, K)
    y = torch.bmm(padded.view(E, largest, K), w.transpose(1, 2).contiguous())
    return y.view(E * largest, N)[place].to(out)


EPS = 1e-6


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import autoround_signsgd_rounding_amd as ar
        if op == "norm":
            r = ar.rmsnorm_fp8(state["x"], state["weight"], EPS, residual=state["residual"],
                               want_y=c["want_y"])
            return {"q": r.q, "scale": r.scale, "h": r.h if c["residual"] else None, "y": r.y}
        if op == "quant_act":
            q, s = ar.fp8_quant_act(state["x"], gate=c["gate"])
            return {"q": q, "scale": s}
        if op == "quant_weight":
            q, s = ar.fp8_quant_weight(state["w"])
            return {"q": q, "scale": s}
        out = DTYPES[c["out"]]
        if op == "gemm":
            return ar.fp8_gemm(state["xq"], state["xs"], state["wq"], state["ws"], out_dtype=out)
        return ar.fp8_gemm_grouped(state["xq"], state["xs"], state["wq"], state["ws"],
                                   state["offsets"], row_index=state["row_index"], out_dtype=out)
    if op == "norm":
        h, y = _norm(state["x"], state["residual"], state["weight"], EPS)
        q, s = _quant_rows(y)
        return {"q": q, "scale": s, "h": h if c["residual"] else None,
                "y": y.to(h.dtype) if c["want_y"] else None}
    if op == "quant_act":
        q, s = _quant_rows(_gated(state["x"]) if c["gate"] else state["x"].float())
        return {"q": q, "scale": s}
    if op == "quant_weight":
        q, s = _quant_weight(state["w"].float())
        return {"q": q, "scale": s}
    out = DTYPES[c["out"]]
    if op == "gemm":
        return _product(state["xq"], state["xs"], state["wq"], state["ws"], out)
    return _grouped_product(state["xq"], state["xs"], state["wq"], state["ws"], state["offsets"],
                            state["row_index"], state["largest"], out)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "norm":
        b = size[case["dtype"]]
        M, D = case["rows"], case["dim"]
        moved = M * D * (b + 1 + (2 * b if case["residual"] else 0) + (b if case["want_y"] else 0))
        return {"bytes": moved + D * b + 4 * M * _blocks(D), "flops": 8 * M * D}
    if op == "quant_act":
        b = size[case["dtype"]]
        M, D = case["rows"], case["dim"]
        return {"bytes": M * D * (b * (2 if case["gate"] else 1) + 1) + 4 * M * _blocks(D),
                "flops": (10 if case["gate"] else 4) * M * D}
    if op == "quant_weight":
        E, N, K = case["experts"], case["rows"], case["dim"]
        return {"bytes": E * N * K * (size[case["dtype"]] + 1) + 4 * E * _blocks(N) * _blocks(K),
                "flops": 4 * E * N * K}
    N, K, b = case["cols"], case["dim"], size[case["out"]]
    if op == "gemm":
        M = case["rows"]
        return {"bytes": (M + N) * K + 4 * (M + _blocks(N)) * _blocks(K) + M * N * b,
                "flops": 2 * M * N * K}
    # an expert without a row is not read: at most as many experts as rows are
    T, R = case["tokens"], case["tokens"] * case["topk"]
    E = min(case["experts"], R)
    X = T if case["gather"] else R
    return {"bytes": X * K + E * N * K + 4 * (X + E * _blocks(N)) * _blocks(K) + R * N * b + 4 * R,
            "flops": 2 * R * N * K}


# ------------------------------------------------------------------ exact values (64 bits)
def _exact_codes(v, amax):
    """Unrounded v / scale and the scale, in 64 bits; amax has v's shape with the blocks spread."""
    s = torch.where(amax == 0, torch.ones_like(amax), (amax / E4M3_MAX).clamp(min=TINY))
    return v / s, s


def _exact_rows(v):
    M, K = v.shape
    q, s = torch.empty_like(v), torch.empty((_blocks(K), M), dtype=v.dtype, device=v.device)
    for j in range(_blocks(K)):
        part = v[:, j * BLOCK:(j + 1) * BLOCK]
        qj, sj = _exact_codes(part, part.abs().max(1, keepdim=True).values)
        q[:, j * BLOCK:(j + 1) * BLOCK], s[j] = qj, sj[:, 0]
    return q, s


def _exact_product(xq, xs, wq, ws):
    """Sum over the 128-wide blocks of xs · ws · (codes · codes), in 64 bits."""
    (M, K), N = xq.shape, wq.shape[0]
    y = torch.zeros((M, N), dtype=torch.float64, device=xq.device)
    n = torch.arange(N, device=xq.device) // BLOCK
    for j in range(_blocks(K)):
        cols = slice(j * BLOCK, min((j + 1) * BLOCK, K))
        p = xq[:, cols].double() @ wq[:, cols].double().t()
        y += p * xs[j].double()[:, None] * ws.double()[n, j][None, :]
    return y


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        x = s["x"].double()
        if case["residual"]:  # the sum is stored, and normalised, in the activations' type
            x = (x + s["residual"].double()).float().to(DTYPES[case["dtype"]]).double()
        ms = (x * x).sum(1) / case["dim"]
        y = x / torch.sqrt(ms + EPS)[:, None] * s["weight"].double()
        q, scale = _exact_rows(y)
        return {"q": q, "scale": scale, "h": x if case["residual"] else None,
                "y": y if case["want_y"] else None}
    if op == "quant_act":
        v = s["x"].double()
        if case["gate"]:
            a, b = v[:, :case["dim"]], v[:, case["dim"]:]
            v = a * torch.sigmoid(a) * b
        q, scale = _exact_rows(v)
        return {"q": q, "scale": scale}
    if op == "quant_weight":
        w = s["w"]
        (E, N, K), q = w.shape, torch.empty(w.shape, dtype=torch.float64, device=w.device)
        scale = torch.empty((E, _blocks(N), _blocks(K)), dtype=torch.float64, device=w.device)
        for i in range(_blocks(N)):
            rows = slice(i * BLOCK, min((i + 1) * BLOCK, N))
            part = w[:, rows].double()
            amax = torch.stack([part[:, :, j * BLOCK:(j + 1) * BLOCK].abs().amax((1, 2))
                                for j in range(_blocks(K))], 1)
            full = amax.repeat_interleave(BLOCK, 1)[:, None, :K].expand_as(part)
            q[:, rows], spread = _exact_codes(part, full)
            scale[:, i] = spread[:, 0, ::BLOCK]
        return {"q": q, "scale": scale}
    if op == "gemm":
        return _exact_product(s["xq"], s["xs"], s["wq"], s["ws"])
    offsets = s["offsets"].tolist()
    y = torch.empty((offsets[-1], case["cols"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        lo, hi = offsets[e], offsets[e + 1]
        if lo < hi:
            rows = s["row_index"][lo:hi].long() if case["gather"] else slice(lo, hi)
            y[lo:hi] = _exact_product(s["xq"][rows], s["xs"][:, rows], s["wq"][e], s["ws"][e])
    return y
