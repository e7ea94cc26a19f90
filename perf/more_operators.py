"""Workloads of the operators around the experts and beside the linears: routing to experts, rows
grouped by expert (or by adapter), the experts' rows added up for each token, and low-rank adapters
of many requests beside a shared projection.

`run` computes an operator in plain torch operations (`own` false) or through the library (`own`
true); `exact` computes it in 64 bits.  Shapes: blocks of 8 to 256 experts, 4096 x 4096 and
4096 x 14336 projections, batches of one token to a prompt of 8192.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEG = float("-inf")


# ------------------------------------------------------------------- cases --

def _route(name, T, E, topk, dtype, score, bias=False, groups=1, topk_groups=1, best=1, renorm=True,
           scale=1.0, masked=0.0):
    return {"name": name, "op": "route", "T": T, "E": E, "topk": topk, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "topk_groups": topk_groups, "best": best, "renorm": renorm,
            "scale": scale, "masked": masked}


def _group(name, T, topk, E, padded=0.0):
    return {"name": name, "op": "group", "T": T, "topk": topk, "E": E, "padded": padded}


def _combine(name, T, topk, N, dtype, residual=False, padded=0.0):
    return {"name": name, "op": "combine", "T": T, "topk": topk, "N": N, "dtype": dtype,
            "residual": residual, "padded": padded}


def _lora(name, M, adapters, rank, K, N, dtype, bare=0.0):
    return {"name": name, "op": "lora", "M": M, "adapters": adapters, "rank": rank, "K": K, "N": N,
            "dtype": dtype, "bare": bare}


def listed():
    return [
        # one decoded token to 8 of 64 experts
        _route("route_t1", 1, 64, 8, "bf16", "softmax"),
        # a ragged prompt, experts that are not a power of two, some of them masked, weights as they are
        _route("route_t1237_masked", 1237, 60, 4, "f16", "softmax", renorm=False, masked=0.05),
        # a prompt of 8192 tokens: sigmoid scores, a bias for balance, 4 of 8 groups
        _route("route_t8192_groups", 8192, 256, 8, "f32", "sigmoid", bias=True, groups=8, topk_groups=4,
               best=2, scale=2.5),
        # a decoding batch of 64 tokens, 8 of 64 experts each
        _group("group_t64", 64, 8, 64),
        # a prompt of 8192 tokens to 8 of 256 experts, padded tokens among them
        _group("group_t8192", 8192, 8, 256, padded=0.03),
        # one decoded token's 8 experts
        _combine("combine_t1", 1, 8, 4096, "bf16"),
        # a ragged prompt, an odd width, slots without an expert, onto the residual stream
        _combine("combine_t1500_odd", 1500, 4, 2003, "f16", residual=True, padded=0.05),
        # a prompt of 8192 tokens, 8 experts each
        _combine("combine_t8192", 8192, 8, 2048, "bf16"),
        # one decoded token with its adapter
        _lora("lora_m1", 1, 4, 16, 4096, 4096, "bf16"),
        # a decoding batch of 64 requests with 32 adapters, a few requests without one
        _lora("lora_m64", 64, 32, 16, 4096, 14336, "bf16", bare=0.1),
        # ragged in every size
        _lora("lora_m777_ragged", 777, 7, 24, 4112, 5001, "f16", bare=0.05),
        # a prompt of 8192 tokens of a few requests, adapters of rank 64
        _lora("lora_m8192", 8192, 4, 64, 4096, 14336, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "group", "combine", "lora"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 384 // groups)
        topk = rng.randint(1, min(12, E))
        topk_groups = rng.randint(1, groups)
        sigmoid = rng.random() < 0.5
        # (groups by their two largest come with the bias, as routers have it)
        best = 2 if sigmoid and groups > 1 else 1
        T = _log(rng, 1, min(16384, 8192 * 256 * 12 // (max(12, 4 + topk) * (E + 2 * topk))))
        c = _route("", T, E, topk, "f32" if sigmoid else dtype, "sigmoid" if sigmoid else "softmax",
                   sigmoid, groups, topk_groups, best, rng.random() < 0.7, rng.choice([1.0, 1.0, 2.5]),
                   rng.choice([0.0, 0.0, 0.05, 0.4]))
    elif op == "group":
        topk = rng.choice([1, 2, 4, 6, 8])
        c = _group("", _log(rng, 1, 65536 // topk), topk, _log(rng, 8, 384), rng.choice([0.0, 0.03, 0.5]))
    elif op == "combine":
        topk = rng.choice([1, 2, 4, 6, 8])
        N = _log(rng, 64, 8192)
        T = _log(rng, 1, min(16384, 8192 * 9 * 2048 // ((4 if dtype == "f32" else 2) * (topk + 2) * N)))
        c = _combine("", T, topk, N, dtype, rng.random() < 0.5, rng.choice([0.0, 0.05, 0.5]))
    else:
        K = 16 * _log(rng, 8, 1024)
        N = _log(rng, 64, 16384)
        rank = 8 * _log(rng, 1, 16)
        M = _log(rng, 1, min(8192, 2 ** 28 // ((4 if dtype == "f32" else 2) * (K + 2 * N))))
        L = _log(rng, 1, min(64, max(1, 2 ** 26 // (rank * (K + N)))))
        c = _lora("", M, L, rank, K, N, dtype, rng.choice([0.0, 0.1, 0.5]))
    del c["name"]
    return c


def work(case):
    op = case["op"]
    if op == "group":
        slots = case["T"] * case["topk"]
        return {"bytes": 4 * slots * 3 + 4 * (case["E"] + 1), "flops": 2 * slots}
    ob = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
    if op == "route":
        T, E, k = case["T"], case["E"], case["topk"]
        return {"bytes": T * E * ob + 8 * T * k + (4 * E if case["bias"] else 0), "flops": T * E * (4 + k)}
    if op == "combine":
        T, k, N = case["T"], case["topk"], case["N"]
        used = T * k * (1.0 - case["padded"])
        rows = used + T * (2 if case["residual"] else 1)
        return {"bytes": rows * N * ob + 8 * T * k, "flops": 2 * used * N}
    M, L, r, K, N = (case[k] for k in ("M", "adapters", "rank", "K", "N"))
    rows = M * (1.0 - case["bare"])
    used = L * (1.0 - (1.0 - 1.0 / L) ** rows)        # adapters that get a row
    return {"bytes": (rows * K + 2 * M * N + used * r * (K + N)) * ob + 4 * (M + L + 1 + used),
            "flops": 2 * rows * r * (K + N)}


# ------------------------------------------------------------------ inputs --

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _choices(g, tokens, topk, experts, padded):
    """Each token's topk distinct experts, some more popular than others; -1 where a slot has none."""
    noise = -torch.log(-torch.log(_uniform(g, tokens, experts) * 0.999 + 5e-4))
    ids = (0.5 * _normal(g, 1, experts) + noise).topk(topk, 1).indices.to(torch.int32)
    return torch.where(_uniform(g, tokens, topk) < padded, -1, ids)


def _order(ids, experts):
    """Slots in the order of their expert (those without one behind), and where each expert's begin."""
    key = torch.where((ids >= 0) & (ids < experts), ids, experts).reshape(-1).long()
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.bincount(key, minlength=experts + 1)[:experts].cumsum(0)
    return torch.argsort(key, stable=True), offsets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    op = case["op"]
    if op == "group":
        s["ids"] = _choices(g, case["T"], case["topk"], case["E"], case["padded"])
        return s
    dt = s["dtype"] = DTYPES[case["dtype"]]
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 1.5 * _normal(g, T, E) + 0.5 * _normal(g, 1, E)
        if case["masked"]:
            # experts that a token may not use; one token in fifty is padding and may use none
            off = (_uniform(g, T, E) < case["masked"]) | (_uniform(g, T, 1) < 0.02)
            logits = torch.where(off, NEG, logits)
        s["logits"] = logits.to(dt)
        s["bias"] = 0.1 * _normal(g, E) if case["bias"] else None
        return s
    if op == "combine":
        T, k, N = case["T"], case["topk"], case["N"]
        experts = max(k, 64)
        ids = _choices(g, T, k, experts, case["padded"])
        order, _ = _order(ids, experts)
        place = torch.empty_like(order)
        place[order] = torch.arange(T * k, device="cuda")
        s["position"] = torch.where(ids >= 0, place.view(T, k), -1).to(torch.int32)
        w = _uniform(g, T, k) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["y"] = (0.5 * _normal(g, T * k, N)).to(dt)
        s["residual"] = _normal(g, T, N).to(dt) if case["residual"] else None
        return s
    M, L, r, K, N = (case[k] for k in ("M", "adapters", "rank", "K", "N"))
    # the plan of the batch: its rows in the order of their adapters, made once for all projections
    ids = _choices(g, M, 1, L, case["bare"])
    order, s["offsets"] = _order(ids, L)
    s["rows"] = order.to(torch.int32)
    s["ends"] = s["offsets"].tolist()             # for the plain form's loop over adapters
    x = _normal(g, M, K)
    s["x"] = torch.where(_uniform(g, M, K) < 0.01, 10.0 * x, x).to(dt)
    s["base"] = _normal(g, M, N).to(dt)           # what the shared projection gave
    s["a"] = (_normal(g, L, r, K) / math.sqrt(K)).to(dt)
    s["b"] = (0.1 * _normal(g, L, N, r)).to(dt)
    s["scales"] = 0.5 + 1.5 * _uniform(g, L)
    return s


# --------------------------------------------------------------- plain form --

def _plain_route(s):
    # the choice in 64 bits: neighbouring scores decide which expert is taken
    case, l = s["case"], s["logits"].double()
    T, E, k, G = case["T"], case["E"], case["topk"], case["groups"]
    top = l.amax(1, keepdim=True)
    top = torch.where(top == NEG, 0.0, top)
    if case["score"] == "softmax":
        e = torch.exp(l - top)
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(l == NEG, NEG, choice)
    if G > 1:
        per = choice.view(T, G, E // G)
        best = per.sort(dim=2, descending=True).values[:, :, :min(case["best"], E // G)]
        value = best[:, :, 0]
        for j in range(1, best.shape[2]):
            value = value + torch.where(best[:, :, j] == NEG, 0.0, best[:, :, j])
        order = value.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device)
        keep.scatter_(1, order, True)
        choice = torch.where(keep[:, :, None], per, NEG).view(T, E)
    value, order = choice.sort(dim=1, descending=True, stable=True)
    value, order = value[:, :k], order[:, :k]
    w = torch.where(value == NEG, 0.0, score.gather(1, order))
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return torch.where(value == NEG, -1, order).to(torch.int32), (w * case["scale"]).float()


def _plain_group(s):
    case, ids = s["case"], s["ids"]
    order, offsets = _order(ids, case["E"])
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    position = torch.where((ids >= 0) & (ids < case["E"]), place.view(ids.shape), -1)
    return (order // case["topk"]).to(torch.int32), offsets, position.to(torch.int32)


def _plain_combine(s):
    y, at = s["y"], s["position"].long()
    rows = y[at.clamp_min(0)].float() * s["weights"][:, :, None]
    out = torch.where((at >= 0)[:, :, None], rows, 0.0).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(s["dtype"])


def _plain_lora(s):
    y, ends, rows = s["base"].clone(), s["ends"], s["rows"].long()
    for e in range(s["case"]["adapters"]):
        if ends[e + 1] > ends[e]:
            at = rows[ends[e]:ends[e + 1]]
            t = s["x"][at].float() @ s["a"][e].float().t()
            d = (t @ s["b"][e].float().t()) * s["scales"][e]
            y[at] = (s["base"][at].float() + d).to(s["dtype"])
    return y


# ------------------------------------------------------------ library calls --

def _own_route(s):
    from bit_groupwise_weight_amd import lowbit as lb
    case = s["case"]
    score = lb.ROUTE_SOFTMAX if case["score"] == "softmax" else lb.ROUTE_SIGMOID
    return lb.lowbit_moe_route(s["logits"], case["topk"], bias=s["bias"], score=score, groups=case["groups"],
                               topk_groups=case["topk_groups"], group_best=case["best"],
                               renormalize=case["renorm"], scale=case["scale"])


def _own_group(s):
    from bit_groupwise_weight_amd import lowbit as lb
    return lb.lowbit_group_rows(s["ids"], s["case"]["E"])


def _own_combine(s):
    from bit_groupwise_weight_amd import lowbit as lb
    return lb.lowbit_moe_combine(s["y"], s["position"], s["weights"], residual=s["residual"])


def _own_lora(s):
    from bit_groupwise_weight_amd import lowbit as lb
    return lb.lowbit_lora(s["x"], s["a"], s["b"], s["scales"], s["rows"], s["offsets"], s["base"])


def run(state):
    op = state["case"]["op"]
    if op == "route":
        return _own_route(state) if own else _plain_route(state)
    if op == "group":
        return _own_group(state) if own else _plain_group(state)
    if op == "combine":
        return _own_combine(state) if own else _plain_combine(state)
    return _own_lora(state) if own else _plain_lora(state)


# ------------------------------------------------------------------- 64 bits --

def _first_largest(v, n):
    """Indices of the n largest of each row in order, the lowest index first among equal ones, and
    their values: one after the other, the chosen ones taken out."""
    v, at, values = v.clone(), [], []
    for _ in range(n):
        m = v.amax(1, keepdim=True)
        i = (v == m).to(torch.uint8).argmax(1, keepdim=True)
        at.append(i)
        values.append(m)
        v.scatter_(1, i, NEG)
    return torch.cat(at, 1), torch.cat(values, 1)


def _exact_route(case, s):
    l = s["logits"].double()
    T, E, k = l.shape[0], l.shape[1], case["topk"]
    dead = torch.isneginf(l)
    if case["score"] == "softmax":
        p = torch.softmax(torch.where(dead.all(1, keepdim=True), 0.0, l), 1)
    else:
        p = torch.sigmoid(l)
    c = p if s["bias"] is None else p + s["bias"].double()
    c = torch.where(dead, NEG, c)
    if case["groups"] > 1:
        per = E // case["groups"]
        values = []
        for q in range(case["groups"]):
            _, v = _first_largest(c[:, q * per:(q + 1) * per], min(case["best"], per))
            rest = torch.where(torch.isneginf(v[:, 1:]), 0.0, v[:, 1:])
            values.append(v[:, 0] + rest.sum(1))
        chosen, _ = _first_largest(torch.stack(values, 1), case["topk_groups"])
        of = torch.arange(E, device=l.device) // per
        c = torch.where((of[None, None, :] == chosen[:, :, None]).any(1), c, NEG)
    at, v = _first_largest(c, k)
    none = torch.isneginf(v)
    w = torch.where(none, 0.0, p.gather(1, at))
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(none, -1, at).to(torch.int32), w * case["scale"]


def _exact_group(case, s):
    ids = s["ids"].reshape(-1).cpu().tolist()
    lists = [[] for _ in range(case["E"] + 1)]
    for slot, e in enumerate(ids):
        lists[e if 0 <= e < case["E"] else case["E"]].append(slot)
    rows, offsets, position = [], [0], [-1] * len(ids)
    for e, slots in enumerate(lists):
        for slot in slots:
            if e < case["E"]:
                position[slot] = len(rows)
            rows.append(slot // case["topk"])
        if e < case["E"]:
            offsets.append(len(rows))

    def up(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    return up(rows), up(offsets), up(position).view(case["T"], case["topk"])


def _exact_combine(case, s):
    out = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
    if s["residual"] is not None:
        out += s["residual"].double()
    for j in range(case["topk"]):
        at = s["position"][:, j]
        has = (at >= 0).nonzero().view(-1)
        out[has] += s["y"][at[has].long()].double() * s["weights"][has, j].double()[:, None]
    return out


def _exact_lora(case, s):
    out = s["base"].double()
    bounds = s["offsets"].cpu().tolist()
    for e, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        a, b = s["a"][e].double().t(), s["b"][e].double().t() * s["scales"][e].double()
        for at in s["rows"][lo:hi].long().split(2048):
            out[at] += (s["x"][at].double() @ a) @ b
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "group": _exact_group, "combine": _exact_combine,
            "lora": _exact_lora}[case["op"]](case, s)
