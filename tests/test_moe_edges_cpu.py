"""F8Experts, MoeRouter and LoraLinear under torch's transforms and at their edges, without a GPU: the
torch layer runs on CPU tensors, with plain stand-ins for the library's calls."""
import warnings

import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn

META = torch.device("meta")
NAN, INF = float("nan"), float("inf")


@pytest.fixture
def calls(monkeypatch):
    """The library's calls in plain torch on CPU tensors; rows that a call leaves undefined are NaN.
    Codes and weights are the numbers themselves, scales are ones.  Returns the names called."""
    seen = []

    def group_rows(ids, E):
        seen.append("group_rows")
        flat = ids.reshape(-1).long()
        key = torch.where((flat >= 0) & (flat < E), flat, E)
        order = torch.argsort(key, stable=True)
        offsets = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
        place = torch.empty_like(order)
        place[order] = torch.arange(order.numel())
        position = torch.where(key < E, place, -1).reshape(ids.shape)
        return ((order // ids.shape[1]).int(), torch.cat([offsets.new_zeros(1), offsets]).int(), position.int())

    def grouped(xq, xscale, offsets, wq, wscale, bias, dtype, rows=None):
        seen.append("linear_f8_grouped")
        T = xq.shape[0] if rows is None else rows.shape[0]
        y = torch.full((T, wq.shape[1]), NAN)
        for e in range(wq.shape[0]):
            at = slice(int(offsets[e]), int(offsets[e + 1]))
            x = xq[at] if rows is None else xq[rows[at].long()]
            y[at] = x.float() @ wq[e].float().t()
        return y.to(dtype)

    def combine(y, position, weights, residual=None):
        seen.append("combine")
        used = (position >= 0).unsqueeze(-1)
        rows = torch.where(used, y[position.clamp(min=0).long()].float(), 0.0)
        return (rows * torch.where(position >= 0, weights, 0.0).unsqueeze(-1)).sum(1).to(y.dtype)

    def quantize(x, xq, xscale):
        xq.copy_(x.clamp(-448, 448))
        xscale.fill_(1.0)

    monkeypatch.setattr(lb, "lowbit_group_rows", group_rows)
    monkeypatch.setattr(lb, "lowbit_linear_f8_grouped", grouped)
    monkeypatch.setattr(lb, "lowbit_moe_combine", combine)
    monkeypatch.setattr(lb, "lowbit_quantize_act_f8", quantize)
    return seen


def experts_of(E=5, H=32, I=16, dtype=torch.float32):
    g = torch.Generator().manual_seed(1)
    m = lnn.F8Experts(E, H, I, dtype=dtype)
    for name, scale in (("gate_up", 1.0), ("down", 1.0)):
        b = getattr(m, name)
        b.copy_((torch.randn(b.shape, generator=g) * scale).to(b.dtype))
    return m


def batch(T=6, E=5, k=3, H=32):
    g = torch.Generator().manual_seed(2)
    e = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)])
    return torch.randn(T, H, generator=g), e, torch.rand(T, k, generator=g), torch.randn(T, k, generator=g)


# ------------------------------------------------ derivatives and batches --

def test_experts_forward_derivative_of_the_routing_weights(calls):
    """The sum is linear in the weights: its tangent is the sum with the tangents for weights."""
    m, (x, e, w, t) = experts_of(), batch()
    e[2, 1] = -1
    want = m(x, e, t)
    assert want.abs().max() > 1
    # (the same products and sums but for their order: a few units of fp32)
    tol = 1e-5 * want.abs().max()
    out, got = torch.func.jvp(lambda w: m(x, e, w), (w,), (t,))
    assert torch.equal(out, m(x, e, w))
    assert (got - want).abs().max() <= tol
    with torch.autograd.forward_ad.dual_level():
        out = m(x, e, torch.autograd.forward_ad.make_dual(w, t))
        assert (torch.autograd.forward_ad.unpack_dual(out).tangent - want).abs().max() <= tol
    # forward and reverse mode, and reverse mode over both: the same derivatives
    fwd, rev = torch.func.jacfwd(lambda w: m(x, e, w))(w), torch.func.jacrev(lambda w: m(x, e, w))(w)
    assert rev.abs().max() > 1 and (fwd - rev).abs().max() <= 1e-5 * rev.abs().max()
    grad = torch.func.grad(lambda w: torch.func.jvp(lambda v: m(x, e, v).square().sum(), (w,), (t,))[1])(w)
    hess = torch.func.hessian(lambda w: m(x, e, w).square().sum())(w)
    assert torch.allclose((hess * t).sum((-1, -2)), grad, rtol=1e-4, atol=1e-4 * grad.abs().max().item())


def test_experts_of_a_batch_of_routing_weights(calls):
    """vmap over the weights is one batched sum, with no fallback to a call a sample."""
    m, (x, e, w, t) = experts_of(), batch()
    ws = torch.stack([w, t, w + t])
    want = torch.stack([m(x, e, v) for v in ws])
    with warnings.catch_warnings():
        warnings.simplefilter("error", UserWarning)
        got = torch.vmap(lambda v: m(x, e, v))(ws)
        tangent = torch.func.jvp(torch.vmap(lambda v: m(x, e, v)), (ws,), (ws,))[1]
        grad = torch.func.grad(lambda ws: torch.vmap(lambda v: m(x, e, v))(ws).sum())(ws)
    assert torch.allclose(got, want, rtol=1e-5, atol=1e-5) and torch.allclose(tangent, want, rtol=1e-5, atol=1e-5)
    assert torch.allclose(grad[0], torch.func.grad(lambda v: m(x, e, v).sum())(w), rtol=1e-5, atol=1e-5)


def test_experts_forward_derivative_on_meta():
    m = lnn.F8Experts(24, 64, 48, device=META)
    x, e = torch.empty(5, 64, dtype=torch.bfloat16, device=META), torch.empty(5, 3, dtype=torch.int32, device=META)
    w = torch.empty(5, 3, device=META)
    with torch.autograd.forward_ad.dual_level():
        out = m(x, e, torch.autograd.forward_ad.make_dual(w, w))
        assert torch.autograd.forward_ad.unpack_dual(out).tangent.shape == (5, 64)


def test_experts_sum_in_the_library_where_no_derivative_is_asked_for(calls):
    m, (x, e, w, t) = experts_of(), batch()
    for run in (lambda: m(x, e, w), lambda: torch.compile(m, fullgraph=True, backend="aot_eager")(x, e, w)):
        del calls[:]
        run()
        assert "combine" in calls
    with torch.no_grad():
        del calls[:]
        m(x, e, w.clone().requires_grad_())
        assert "combine" in calls
    for run in (lambda: m(x, e, w.clone().requires_grad_()), lambda: torch.func.jvp(lambda v: m(x, e, v), (w,), (t,))):
        del calls[:]
        run()
        assert calls and "combine" not in calls


def test_compiled_experts_keep_their_derivatives(calls):
    m, (x, e, w, t) = experts_of(), batch()
    for fn in (lambda w, t: torch.func.jvp(lambda v: m(x, e, v), (w,), (t,))[1],
               lambda w, t: torch.func.grad(lambda v: m(x, e, v).sum())(w),
               lambda w, t: torch.vmap(lambda v: m(x, e, v))(torch.stack([w, t]))):
        torch._dynamo.reset()
        want = fn(w, t)
        got = torch.compile(fn, fullgraph=True, backend="aot_eager")(w, t)
        assert want.abs().max() > 1 and (got - want).abs().max() <= 1e-5 * want.abs().max()


# ----------------------------------------------------------- padded slots --

def test_experts_gradient_beside_rows_that_are_not_finite(calls):
    """A token that is not finite, whose rows come first, leaves the gradients of other tokens' padded
    slots alone: they are 0, and the other weights' are what they are without it."""
    m, (x, e, w, up) = experts_of(), batch()
    up = torch.randn(6, 32, generator=torch.Generator().manual_seed(3))
    e[0] = torch.tensor([0, 1, 2])                      # row 0 of the experts' is token 0's
    e[2, 1], e[4, 0], e[4, 2] = -1, 5, -1

    def grad(x):
        v = w.clone().requires_grad_()
        out = m(x, e, v)
        (out * torch.where(torch.arange(6)[:, None] > 0, up, 0.0))[1:].sum().backward()
        return out.detach(), v.grad

    out, want = grad(x)
    for bad in (NAN, INF):
        y = x.clone()
        y[0] = bad
        got_out, got = grad(y)
        assert torch.equal(got_out[1:], out[1:])
        assert torch.equal(got[1:], want[1:])
        assert got[2, 1] == 0 and got[4, 0] == 0 and got[4, 2] == 0
    assert want[1].abs().min() > 0


def test_experts_gradient_where_no_slot_has_an_expert(calls):
    """Nothing is written for any row then: sums and gradients are 0, whatever the weights hold."""
    m, (x, e, w, _) = experts_of(), batch()
    e[:] = -1
    for fill in (1.0, NAN, INF):
        v = torch.full_like(w, fill).requires_grad_()
        out = m(x, e, v)
        assert (out == 0).all() and torch.equal(out.detach(), m(x, e, v.detach()))
        out.sum().backward()
        assert (v.grad == 0).all()


@pytest.mark.parametrize("weight", [NAN, INF, -INF])
def test_experts_padded_slots_of_any_weight_add_nothing(calls, weight):
    m, (x, e, w, t) = experts_of(), batch()
    e[3, 2] = -1
    w[3, 2] = weight
    plain = m(x, e, w)
    assert torch.isfinite(plain).all()
    v = w.clone().requires_grad_()
    out = m(x, e, v)
    assert torch.allclose(out, plain, rtol=1e-5, atol=1e-5)
    out.sum().backward()
    assert torch.isfinite(v.grad).all() and v.grad[3, 2] == 0
    assert torch.isfinite(torch.func.jvp(lambda u: m(x, e, u), (w,), (t,))[1]).all()


def test_experts_of_very_many_slots_keep_torch_s_order_of_the_sum(calls):
    """torch's sum over up to 31 slots is the library's, bit for bit; from 32 on it adds in another
    order, and is kept."""
    m = experts_of(E=40)
    for k in (31, 32, 40):
        x, e, w, _ = batch(E=40, k=k)
        del calls[:]
        m(x, e, w)
        assert ("combine" in calls) == (k < 32)


@pytest.mark.parametrize("shape", [(6,), (2, 3), (0,)])
def test_experts_of_no_slots_are_zeros(calls, shape):
    m = experts_of(dtype=torch.bfloat16)
    x = torch.randn(*shape, 32).bfloat16()
    e, w = torch.empty(*shape, 0, dtype=torch.int32), torch.empty(*shape, 0)
    out = m(x, e, w)
    assert out.shape == x.shape and out.dtype == torch.bfloat16 and (out == 0).all()
    v = w.clone().requires_grad_()
    m(x, e, v).float().sum().backward()
    assert v.grad.shape == v.shape
    meta = lnn.F8Experts(5, 32, 16, device=META)
    out = meta(x.to(META), e.to(META), w.to(META))
    assert out.shape == x.shape and out.device == META


# ------------------------------------------- modules without a derivative --

def router_and_lora(monkeypatch):
    def route(logits, topk, bias, *rest):
        w, e = torch.softmax(logits.float(), -1).topk(topk, -1)
        return e.int(), w

    def lora(x, a, b, scales, rows, offsets, base, y=None):
        y = base.clone() if y is None else y
        for l in range(a.shape[0]):
            at = rows[int(offsets[l]):int(offsets[l + 1])].long()
            y[at] = (base[at].float() + (x[at].float() @ a[l].float().t()) @ b[l].float().t() * scales[l]).to(y.dtype)
        return y

    monkeypatch.setattr(lb, "lowbit_moe_route", route)
    monkeypatch.setattr(lb, "lowbit_lora", lora)
    g = torch.Generator().manual_seed(5)
    m = lnn.LoraLinear(torch.nn.Linear(32, 24), 2, 8).requires_grad_(False)
    for i in range(2):
        m.set_adapter(i, torch.randn(8, 32, generator=g), torch.randn(24, 8, generator=g), 0.5)
    return lnn.MoeRouter(12, 3, bias=True), m, torch.randn(5, 12, generator=g), torch.randn(5, 32, generator=g)


def test_router_and_adapters_refuse_forward_mode(calls, monkeypatch):
    """They have no derivative: reverse mode raises at the backward pass, forward mode at the call, where
    the tangent would be dropped without a word."""
    router, m, logits, x = router_and_lora(monkeypatch)
    plan = lnn.adapter_plan(torch.tensor([0, 1, -1, 1, 0]), 2)
    route = lambda l: router(l)[1]
    adapt = lambda v: m(v, plan)
    for f, v in ((route, logits), (adapt, x)):
        for g in (lambda: torch.func.jvp(f, (v,), (v,)), lambda: torch.func.jacfwd(f)(v),
                  lambda: torch.vmap(lambda u: torch.func.jvp(f, (u,), (u,)))(v[None]),
                  lambda: torch.func.jvp(torch.vmap(f), (v[None],), (v[None],)),
                  lambda: torch.func.jvp(lambda a: torch.func.jvp(f, (a,), (v,))[1], (v,), (v,)),
                  lambda: torch.compile(lambda u: torch.func.jvp(f, (u,), (u,))[1], backend="eager")(v)):
            with pytest.raises(RuntimeError, match="forward"):
                g()
        with torch.autograd.forward_ad.dual_level(), pytest.raises(RuntimeError, match="forward"):
            f(torch.autograd.forward_ad.make_dual(v, v))
        with pytest.raises(RuntimeError):
            f(v.clone().requires_grad_()).sum().backward()
        with pytest.raises(RuntimeError):
            torch.func.grad(lambda u: f(u).sum())(v)
    with pytest.raises(RuntimeError, match="forward"):
        torch.func.jvp(lambda a: torch.func.functional_call(m, {"a": a}, (x, plan)), (m.a,), (m.a,))


def test_router_and_adapters_beside_a_derivative_of_something_else(calls, monkeypatch):
    """Tensors without a tangent pass, inside a forward-mode derivative and under vmap."""
    router, m, logits, x = router_and_lora(monkeypatch)
    plan = lnn.adapter_plan(torch.tensor([0, 1, -1, 1, 0]), 2)
    w, y = router(logits)[1], m(x, plan)
    t = torch.ones(3)
    out, tangent = torch.func.jvp(lambda s: s * router(logits)[1], (t,), (t,))
    assert torch.equal(out, w) and torch.equal(tangent, w)
    out, tangent = torch.func.jvp(lambda s: s[0] * m(x, plan), (t,), (t,))
    assert torch.equal(out, y) and torch.equal(tangent, y)
    # no plan, no adapters: the linear's own derivative
    assert torch.equal(torch.func.jvp(m, (x,), (x,))[1], x @ m.linear.weight.t())
    fn = torch.compile(lambda l, v: (router(l)[1], m(v, plan)), fullgraph=True, backend="aot_eager")
    got = fn(logits, x)
    assert torch.equal(got[0], w) and torch.equal(got[1], y)
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        assert torch.equal(torch.vmap(lambda l: router(l)[1])(logits[None])[0], w)


# ------------------------------------------------------- modules, moved ----

@pytest.mark.parametrize("make", [
    lambda: lnn.LoraLinear(torch.nn.Linear(32, 24, device=META, dtype=torch.bfloat16), 2, 8),
    lambda: lnn.LoraLinear(lnn.F8Linear(32, 24, device=META), 2, 8),
    lambda: lnn.MoeRouter(12, 3, bias=True, device=META),
])
def test_modules_built_on_meta_are_materialized(make):
    m = make().to_empty(device="cpu")
    assert all(t.device.type == "cpu" for t in (*m.buffers(), *m.parameters()))
    kept = m.scales if isinstance(m, lnn.LoraLinear) else m.bias
    assert kept.dtype == torch.float32
    kept.fill_(0.1)
    m = m.half()
    kept = m.scales if isinstance(m, lnn.LoraLinear) else m.bias
    assert kept.dtype == torch.float32 and (kept == torch.tensor(0.1)).all()


def test_lora_linear_keeps_its_scales_through_casts_and_moves():
    """Their values and type; what the move itself does to them (here: memory of their own) is kept."""
    m = lnn.LoraLinear(torch.nn.Linear(32, 24), 3, 8)
    m.scales.copy_(torch.tensor([0.1, 1e-30, 3.0]))
    want = m.scales.clone()
    for cast in (lambda m: m.bfloat16(), lambda m: m.to(torch.float16), lambda m: m.double(), lambda m: m.float(),
                 lambda m: m.cpu()):
        m = cast(m)
        assert m.scales.dtype == torch.float32 and torch.equal(m.scales, want)
    before = m.scales
    m._apply(lambda t: t.clone())
    assert torch.equal(m.scales, want) and m.scales.data_ptr() != before.data_ptr()
    assert torch.equal(lnn.LoraLinear(torch.nn.Linear(32, 24), 3, 8).share_memory().scales, torch.ones(3))


def test_router_names_all_its_settings():
    text = repr(lnn.MoeRouter(24, 3, "sigmoid", bias=True, groups=4, topk_groups=2, group_best=2, renormalize=False,
                              scale=2.5))
    for part in ("num_experts=24", "topk=3", "score=sigmoid", "bias=True", "groups=4", "topk_groups=2", "group_best=2",
                 "renormalize=False", "scale=2.5"):
        assert part in text


# ---------------------------------------------------- rows that are named ----

@pytest.fixture
def lora_calls(monkeypatch):
    """lowbit_lora in plain torch: only rows that `rows` names are written; y of the call's own is NaN."""
    seen = []

    def lora(x, a, b, scales, rows, offsets, base, y=None):
        seen.append("fresh" if y is None else "given")
        M, L = x.shape[0], a.shape[0]
        y = torch.full((M, b.shape[1]), NAN, dtype=x.dtype) if y is None else y
        was = torch.zeros_like(y) if base is None else base.clone()
        at = torch.arange(M) if rows is None else rows.long()
        for p, m in enumerate(at.tolist()):
            if not 0 <= m < M:
                continue
            l = next((l for l in range(L) if offsets[l] <= p < offsets[l + 1]), None)
            y[m] = was[m]
            if l is not None:
                y[m] += (x[m] @ a[l].t()) @ b[l].t() * (1.0 if scales is None else scales[l])
        return y

    monkeypatch.setattr(lb, "lowbit_lora", lora)
    return seen


@pytest.mark.parametrize("with_base", [False, True])
@pytest.mark.parametrize("rows, offsets", [
    ([3, -1, 0, 6, 2, 9], [0, 3, 5]),            # as many as there are rows, some of them none
    ([-1] * 6, [0, 3, 6]),
    ([3, 1, -1, -1, -1, -1, -1, -1], [0, 1, 2]),  # more: a plan of fixed length, filled up
    ([3, 1], [0, 1, 2]), ([], [0, 0, 0]),        # fewer
    ([5, 4, 3, 2, 1, 0], [0, 2, 4]),             # all of them
])
def test_op_lora_keeps_base_in_rows_that_are_not_named(lora_calls, with_base, rows, offsets):
    g = torch.Generator().manual_seed(4)
    x, a, b = torch.randn(6, 32, generator=g), torch.randn(2, 8, 32, generator=g), torch.randn(2, 24, 8, generator=g)
    base = torch.randn(6, 24, generator=g) if with_base else None
    kept = base.clone() if with_base else None
    y = torch.ops.lowbit.lora(x, a, b, None, torch.tensor(rows, dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32), base)
    assert torch.isfinite(y).all()
    was = torch.zeros(6, 24) if base is None else base
    want = was.clone()
    for p, m in enumerate(rows):
        l = 0 if p < offsets[1] else 1 if p < offsets[2] else None
        if 0 <= m < 6 and l is not None and p >= offsets[0]:
            want[m] += (x[m] @ a[l].t()) @ b[l].t()
    assert torch.equal(y, want)
    assert base is None or torch.equal(base, kept)


def test_lora_linear_takes_plans_of_other_makers(lora_calls, calls):
    """adapter_plan's names every row, and no copy of the linear's output is made for it; any other
    plan's rows that are not named keep the linear's output."""
    m = lnn.LoraLinear(torch.nn.Linear(32, 24), 2, 8).requires_grad_(False)
    for i in range(2):
        m.set_adapter(i, torch.randn(8, 32), torch.randn(24, 8))
    x = torch.randn(2, 3, 32)
    plan = lnn.adapter_plan(torch.tensor([0, 1, 1, -1, 0, 1]), 2)
    rows, offsets = plan
    y = m(x, plan)
    assert lora_calls == ["fresh"]
    assert torch.equal(y, m(x, (rows, offsets))) and lora_calls == ["fresh", "given"]
    own = m(x, (torch.tensor([1, -1, 8, 4, -1, -1], dtype=torch.int32), torch.tensor([0, 1, 4], dtype=torch.int32)))
    base = m.linear(x)
    assert torch.equal(own.view(6, 24)[[0, 2, 3, 5]], base.view(6, 24)[[0, 2, 3, 5]])
    assert not torch.equal(own, base) and torch.isfinite(own).all()
    # (as many entries as rows: only the maker's word tells a whole plan from another)
    del lora_calls[:]
    m(x, lnn.AdapterPlan(rows, offsets))
    fn = torch.compile(m, fullgraph=True, backend="aot_eager")
    assert torch.equal(fn(x, plan), y) and lora_calls == ["fresh", "fresh"]


def test_ops_take_strided_plans_scales_and_weights(lora_calls, calls, monkeypatch):
    """Any strides, as of the other arguments: what reaches the library is contiguous."""
    seen = []
    for name in ("lowbit_lora", "lowbit_linear_f8_grouped", "lowbit_moe_combine"):
        def call(*args, _run=getattr(lb, name), **kw):
            seen.extend(t.is_contiguous() for t in (*args, *kw.values()) if torch.is_tensor(t))
            return _run(*args, **kw)
        monkeypatch.setattr(lb, name, call)
    wide = lambda t: torch.stack([t, t], -1)[..., 0]
    x, a, b = torch.randn(6, 32), torch.randn(2, 8, 32), torch.randn(2, 24, 8)
    rows, offsets = torch.arange(6).int(), torch.tensor([0, 2, 5]).int()
    args = (x, a, b, torch.rand(2), rows, offsets, torch.randn(6, 24))
    assert torch.equal(torch.ops.lowbit.lora(*map(wide, args)), torch.ops.lowbit.lora(*args))
    position, w = torch.tensor([[0, 1], [3, -1]]).int(), torch.rand(2, 2)
    args = (x, position, w, torch.randn(2, 32))
    assert torch.equal(torch.ops.lowbit.moe_combine(*map(wide, args)),
                       torch.ops.lowbit.moe_combine(*args))
    assert seen and all(seen)


@pytest.mark.parametrize("call", [
    lambda m: torch.ops.lowbit.lora(m(4, 32), m(3, 8, 32), m(3, (1 << 23) + 1, 8), None, None, m(4, dtype=torch.int32), None),
    lambda m: torch.ops.lowbit.lora(m(4, (1 << 23) + 16), m(3, 8, (1 << 23) + 16), m(3, 40, 8), None, None,
                                    m(4, dtype=torch.int32), None),
    lambda m: torch.ops.lowbit.lora(m(4, 32), m(65537, 8, 32), m(65537, 40, 8), None, None, m(65538, dtype=torch.int32), None),
    lambda m: torch.ops.lowbit.moe_route(m(4, 8), None, 2, 0, 1, 1, 1, True, INF),
    lambda m: torch.ops.lowbit.moe_combine(m(4, 8), m(2, 65537, dtype=torch.int32), m(2, 65537), None),
])
def test_shape_functions_refuse_sizes_that_the_calls_refuse(call):
    """(Not numbers of rows, which a compiled program may not know.)"""
    with pytest.raises(ValueError):
        call(lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device=META))


def test_group_rows_needs_no_workspace_up_to_its_bounds(lowbit_lib):
    """What the binding leaves unasked: up to that many slots and experts the library asks for none."""
    need = lowbit_lib.lowbit_group_rows_workspace_bytes
    for E in (1, 64, lb.GROUP_ROWS_EXPERTS):
        for k in (1, 3, 8):
            assert need(lb.GROUP_ROWS_ALONE // k, k, E) == 0
        assert need(lb.GROUP_ROWS_ALONE + 1, 1, E) > 0
    assert need(lb.GROUP_ROWS_ALONE, 1, 65536) > 0


@pytest.mark.parametrize("E", [1, 64, 900, 901, 4096, 65536])
def test_group_rows_workspace_grows_with_the_slots(lowbit_lib, E):
    """At most a few bytes a slot, up to the largest call: counts of chunks, and two copies of the slots
    where the experts are many."""
    need = lowbit_lib.lowbit_group_rows_workspace_bytes
    for p in range(0, 31):
        assert need(1 << p, 1, E) <= (1 << p) * 12 + 4 * 128 * (E if E <= 900 else 512) + 8192
    assert need(1 << 30, 1, E) > 0 and need((1 << 30) + 1, 1, E) == 0


def test_experts_in_inference_mode(calls):
    m, (x, e, w, _) = experts_of(), batch()
    want = m(x, e, w)
    with torch.inference_mode():
        del calls[:]
        assert torch.equal(m(x, e, w), want) and torch.equal(m(x, e, w.clone()), want) and "combine" in calls
