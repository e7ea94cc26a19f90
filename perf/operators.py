"""Workloads of the 8-bit operators: the residual-add RMS norm with 8-bit output, the fp8 linear
with a scale for each block of 128, and the fp8 linear grouped by expert.

`run` computes an operator in plain torch operations (`own` false) or through the library (`own`
true); `exact` computes it in 64 bits.  Shapes: Llama-3.1-8B-shaped linears (4096 x 4096,
4096 x 14336, 14336 x 4096, batch 1 and 128) and generic mixture-of-experts blocks.
"""
import math

import torch

own = False

BLOCK = 128                 # K elements that share a scale (and weight rows that do)
E4M3_MAX = 448.0
EPS = 1e-5
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases --

def _norm(name, M, K, dtype, fmt, residual=True, want_y=False):
    return {"name": name, "op": "norm", "M": M, "K": K, "dtype": dtype, "fmt": fmt,
            "residual": residual, "want_y": want_y}


def _linear(name, M, K, N, dtype, bias=False):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "dtype": dtype, "bias": bias}


def _grouped(name, tokens, topk, experts, K, N, dtype, gather, pad=0, bias=False):
    return {"name": name, "op": "grouped", "tokens": tokens, "topk": topk, "experts": experts,
            "K": K, "N": N, "dtype": dtype, "gather": gather, "pad": pad, "bias": bias}


def listed():
    return [
        # one decoded token's hidden state before its projections
        _norm("norm_m1_f8", 1, 4096, "bf16", "f8"),
        # a batch of 128 into the int8-activation linear (its 14336-wide input)
        _norm("norm_m128_i8", 128, 14336, "bf16", "i8", residual=False),
        # an odd number of rows, a last block of 32, fp16; the router reads y
        _norm("norm_m1237_f8_y", 1237, 2080, "f16", "f8", want_y=True),
        # a prompt of 8192 tokens
        _norm("norm_m8192_f8", 8192, 4096, "bf16", "f8"),
        # one decoded token: the up projection
        _linear("linear_m1", 1, 4096, 14336, "bf16"),
        # the batch of 128: the down projection
        _linear("linear_m128", 128, 14336, 4096, "bf16"),
        # ragged in every size, with a bias
        _linear("linear_m777_ragged", 777, 4112, 5000, "f16", bias=True),
        # a prompt of 8192 tokens: the up projection
        _linear("linear_m8192", 8192, 4096, 14336, "bf16"),
        # one decoded token to 8 of 64 experts
        _grouped("grouped_t1", 1, 8, 64, 4096, 2048, "bf16", gather=True),
        # a decoding batch of 64: 8 rows an expert on average, some experts with none
        _grouped("grouped_t64", 64, 8, 64, 2048, 1408, "bf16", gather=True),
        # the down projection of a ragged prompt: rows already grouped, rows behind the last group
        _grouped("grouped_t1500_pad", 1500, 4, 16, 1424, 2000, "f16", gather=False, pad=77, bias=True),
        # a prompt of 8192 tokens to 2 of 8 experts
        _grouped("grouped_t8192", 8192, 2, 8, 4096, 4096, "bf16", gather=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "grouped"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        fmt = rng.choice(["f8", "i8"])
        unit = 32 if fmt == "i8" else 16
        K = unit * _log(rng, 4, 16384 // unit)
        M = _log(rng, 1, min(16384, 8192 * 4096 // K))
        c = _norm("", M, K, dtype, fmt, rng.random() < 0.7, rng.random() < 0.3)
    elif op == "linear":
        K = 16 * _log(rng, 8, 1024)
        N = _log(rng, 64, 16384)
        M = _log(rng, 1, min(8192, 8192 * 4096 * 14336 // (4 * N * K)))
        c = _linear("", M, K, N, dtype, rng.random() < 0.5)
    else:
        E = rng.choice([4, 8, 16, 32, 64, 128])
        topk = rng.choice([1, 2, 4])
        K = 16 * _log(rng, 8, 512)
        N = _log(rng, 64, min(8192, 2 ** 29 // (E * K)))
        tokens = _log(rng, 1, min(8192, 8192 * 2 * 4096 * 4096 // (4 * topk * N * K)))
        c = _grouped("", tokens, topk, E, K, N, dtype, rng.random() < 0.5, rng.choice([0, 0, 13]),
                     rng.random() < 0.3)
    del c["name"]
    return c


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    K, ob = case["K"], torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
    kb = _blocks(K)
    if case["op"] == "norm":
        M = case["M"]
        scales = 4 * M * (kb if case["fmt"] == "f8" else 1)
        per = ob + 1 + (2 * ob if case["residual"] else 0) + (ob if case["want_y"] else 0)
        return {"bytes": M * K * per + scales + K * ob, "flops": 8 * M * K}
    N, bias = case["N"], ob if case["bias"] else 0
    if case["op"] == "linear":
        M = case["M"]
        b = M * (K + 4 * kb) + N * K + 4 * _blocks(N) * kb + M * N * ob + N * bias
        return {"bytes": b, "flops": 2 * M * N * K}
    E, tokens, T = case["experts"], case["tokens"], case["tokens"] * case["topk"]
    used = E * (1.0 - (1.0 - case["topk"] / E) ** tokens)       # experts that get a row
    rows = tokens if case["gather"] else T
    b = rows * (K + 4 * kb) + used * (N * K + 4 * _blocks(N) * kb + N * bias) + T * N * ob
    b += 4 * (E + 1) + (4 * T if case["gather"] else 0)
    return {"bytes": b, "flops": 2 * T * N * K}


# ------------------------------------------------------------------ inputs --

def _activations(g, M, K):
    """N(0, 1) with one value in a hundred twenty times as large."""
    x = torch.randn(M, K, generator=g, device="cuda")
    big = torch.rand(M, K, generator=g, device="cuda") < 0.01
    return torch.where(big, 20.0 * x, x)


def _codes_of_rows(x):
    """e4m3 codes of x[M, K] and the scale of each block of 128 of a row."""
    M, K = x.shape
    kb = _blocks(K)
    p = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    s = p.abs().amax(2) / E4M3_MAX
    q = (p / s.clamp_min(1e-30)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(M, -1)[:, :K].contiguous().view(torch.float8_e4m3fn), s


def _weights(g, N, K):
    """e4m3 codes of a weight whose rows have standard deviations in [0.005, 0.05], and the scale
    of each block of 128 x 128."""
    lo, hi = math.log(0.005), math.log(0.05)
    sd = torch.exp(lo + (hi - lo) * torch.rand(N, 1, generator=g, device="cuda"))
    w = torch.randn(N, K, generator=g, device="cuda") * sd
    nb, kb = _blocks(N), _blocks(K)
    p = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    s = p.abs().amax((1, 3)) / E4M3_MAX
    q = (p / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).view(nb * BLOCK, kb * BLOCK)[:N, :K].contiguous()
    return q.view(torch.float8_e4m3fn), s


def _routing(g, tokens, topk, experts):
    """Each token's topk distinct experts, some experts more popular than others: the tokens in
    order of their experts, and where each expert's rows begin."""
    like = 0.5 * torch.randn(1, experts, generator=g, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, generator=g, device="cuda") * 0.999 + 5e-4))
    ids = (like + noise).topk(topk, 1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return (order // topk).to(torch.int32), offsets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, K = DTYPES[case["dtype"]], case["K"]
    s = {"case": case, "dtype": dt}
    if case["op"] == "norm":
        M = case["M"]
        s["x"] = _activations(g, M, K).to(dt)
        s["residual"] = (3.0 * torch.randn(M, K, generator=g, device="cuda")).to(dt) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(dt)
        if case["fmt"] == "i8":
            s["values"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        return s
    N = case["N"]
    if case["op"] == "linear":
        s["xq"], s["xs"] = _codes_of_rows(_activations(g, case["M"], K))
        s["wq"], s["ws"] = _weights(g, N, K)
        s["bias"] = (0.1 * torch.randn(N, generator=g, device="cuda")).to(dt) if case["bias"] else None
        return s
    E, T = case["experts"], case["tokens"] * case["topk"]
    rows, s["offsets"] = _routing(g, case["tokens"], case["topk"], E)
    s["rows"] = rows if case["gather"] else None
    s["ends"] = s["offsets"].tolist()             # for the plain form's loop over experts
    total = T + case["pad"]                       # a padded batch: rows that belong to no expert
    if case["gather"] and case["pad"]:
        s["rows"] = torch.cat([rows, rows.new_zeros(case["pad"])])
    s["xq"], s["xs"] = _codes_of_rows(_activations(g, case["tokens"] if case["gather"] else total, K))
    per = [_weights(g, N, K) for _ in range(E)]
    s["wq"] = torch.stack([q.view(torch.uint8) for q, _ in per]).view(torch.float8_e4m3fn)
    s["ws"] = torch.stack([w for _, w in per])
    s["bias"] = (0.1 * torch.randn(E, N, generator=g, device="cuda")).to(dt) if case["bias"] else None
    s["y"] = torch.zeros(total, N, dtype=dt, device="cuda")
    return s


# --------------------------------------------------------------- plain form --

def _spread_rows(s, K):
    return s.repeat_interleave(BLOCK, 1)[:, :K]


def _dequant_rows(q, s):
    return q.float() * _spread_rows(s, q.shape[1])


def _dequant_weight(q, s):
    N, K = q.shape
    return q.float() * _spread_rows(s, K).repeat_interleave(BLOCK, 0)[:N]


def _plain_norm(s):
    case, x, K = s["case"], s["x"].float(), s["case"]["K"]
    h = x if s["residual"] is None else (x + s["residual"].float()).to(s["dtype"]).float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    out = {}
    if s["residual"] is not None:
        out["sum"] = h.to(s["dtype"])
    if case["want_y"]:
        out["y"] = y.to(s["dtype"])
    if case["fmt"] == "i8":
        a = y.abs().amax(1) / 127.0
        q = torch.round(y / a[:, None]).clamp(-127.0, 127.0)
        out["values"], out["scale"] = (q * a[:, None]).to(torch.bfloat16), a
    else:
        kb = _blocks(K)
        p = torch.nn.functional.pad(y, (0, kb * BLOCK - K)).view(-1, kb, BLOCK)
        scale = p.abs().amax(2) / E4M3_MAX
        q = (p / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        out["values"] = q.view(-1, kb * BLOCK)[:, :K].to(torch.float8_e4m3fn)
        out["scale"] = scale
    return out


def _plain_linear(s):
    y = _dequant_rows(s["xq"], s["xs"]) @ _dequant_weight(s["wq"], s["ws"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["dtype"])


def _plain_grouped(s):
    x = _dequant_rows(s["xq"], s["xs"])
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    ends, y = s["ends"], s["y"]
    for e in range(s["case"]["experts"]):
        if ends[e + 1] > ends[e]:
            part = x[ends[e]:ends[e + 1]] @ _dequant_weight(s["wq"][e], s["ws"][e]).t()
            if s["bias"] is not None:
                part = part + s["bias"][e].float()
            y[ends[e]:ends[e + 1]] = part.to(s["dtype"])
    return y


# ------------------------------------------------------------ library calls --

def _own_norm(s):
    from bit_groupwise_weight_amd import lowbit as lb
    case = s["case"]
    fmt = lb.Q8_I8 if case["fmt"] == "i8" else lb.Q8_F8
    q, scale, total, y = lb.lowbit_add_rmsnorm_q8(s["x"], s["weight"], EPS, fmt, residual=s["residual"],
                                                  want_y=case["want_y"])
    out = {"scale": scale}
    if total is not None:
        out["sum"] = total
    if y is not None:
        out["y"] = y
    # int8 codes as the values they stand for (e4m3 codes are floating-point numbers as they are)
    out["values"] = q if case["fmt"] == "f8" else torch.mul(q, scale[:, None], out=s["values"])
    return out


def _own_linear(s):
    from bit_groupwise_weight_amd import lowbit as lb
    return lb.lowbit_linear_f8(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"], s["dtype"])


def _own_grouped(s):
    from bit_groupwise_weight_amd import lowbit as lb
    return lb.lowbit_linear_f8_grouped(s["xq"], s["xs"], s["offsets"], s["wq"], s["ws"], s["bias"],
                                       s["dtype"], rows=s["rows"], y=s["y"])


def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    if op == "linear":
        return _own_linear(state) if own else _plain_linear(state)
    return _own_grouped(state) if own else _plain_grouped(state)


# ------------------------------------------------------------------- 64 bits --

def _nearest_e4m3(v):
    """v rounded to the nearest number of 4 significant bits, exponents down to -6, ties to even."""
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -6))
    step = torch.ldexp(torch.ones_like(v), e - 4)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _matmul64(xq, xs, wq, ws):
    """Sum over blocks of scale * scale * (exact sum of code products), in float64."""
    K = xq.shape[1]
    total = None
    x, w = xq.double(), wq.double()
    cols = torch.arange(K, device=x.device) // BLOCK
    rows = torch.arange(w.shape[0], device=x.device) // BLOCK
    x = x * xs.double()[:, cols]
    w = w * ws.double()[rows][:, cols]
    for k in range(0, K, 4096):
        part = x[:, k:k + 4096] @ w[:, k:k + 4096].t()
        total = part if total is None else total + part
    return total


def exact(case, seed):
    s = prepare(case, seed)
    K = case["K"]
    if case["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (s["x"].double() + s["residual"].double()).float().to(s["dtype"]).double()
        y = h / torch.sqrt((h ** 2).sum(1, keepdim=True) / K + EPS) * s["weight"].double()
        out = {}
        if s["residual"] is not None:
            out["sum"] = h
        if case["want_y"]:
            out["y"] = y
        if case["fmt"] == "i8":
            a = y.abs().max(1).values / 127
            out["values"], out["scale"] = torch.round(y / a[:, None]) * a[:, None], a
        else:
            full = torch.zeros(case["M"], _blocks(K) * BLOCK, dtype=torch.float64, device=y.device)
            full[:, :K] = y
            out["scale"] = full.view(case["M"], -1, BLOCK).abs().max(2).values / E4M3_MAX
            out["values"] = _nearest_e4m3(y / out["scale"].repeat_interleave(BLOCK, 1)[:, :K])
        return out
    if case["op"] == "linear":
        y = _matmul64(s["xq"], s["xs"], s["wq"], s["ws"])
        return y if s["bias"] is None else y + s["bias"].double()
    x = s["xq"].view(torch.uint8)
    xs = s["xs"]
    if s["rows"] is not None:
        x, xs = x[s["rows"].long()], xs[s["rows"].long()]
    x = x.view(torch.float8_e4m3fn)
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=x.device)
    ends = s["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            y[a:b] = _matmul64(x[a:b], xs[a:b], s["wq"][e], s["ws"][e])
            if s["bias"] is not None:
                y[a:b] += s["bias"][e].double()
    return y
