"""F8Experts and the operators around the experts on the GPU, at their edges: derivatives in every
mode, the sum's equality with torch's, orders and choices that the other tests' shapes do not reach."""
import numpy as np
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn
from oracle import moe_oracle as o

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
NEG, INF, NAN = float("-inf"), float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _lib(lowbit_lib):
    return lowbit_lib


def f64(t):
    return t.detach().double().cpu().numpy()


def experts_of(seed, E=6, H=64, I=48, dtype=torch.float32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def n(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    m = lnn.F8Experts(E, H, I, dtype=dtype, device=DEV).set_weight(n(E, 2 * I, H) * 0.1, n(E, H, I) * 0.1)
    return m, n, g


# -------------------------------------------------------------- derivatives --

def test_experts_forward_and_reverse_derivatives_agree():
    """The sum is linear in the routing weights.  Its tangent is the sum with the tangents for weights
    and its Jacobian's columns are the slots' rows: products and sums of three terms in fp32, each
    rounded once, on either side (2 * 4 * 2^-24 of the terms' magnitudes)."""
    m, n, g = experts_of(21)
    x, w, t = n(9, 64), n(9, 3), n(9, 3)
    e = torch.stack([torch.randperm(6, generator=g, device=DEV)[:3] for _ in range(9)])
    e[2, 1] = -1
    size = 8 * U * m(x, e, t.abs()).abs().max() * 3
    want = m(x, e, t)
    assert want.abs().max() > 0
    out, tangent = torch.func.jvp(lambda w: m(x, e, w), (w,), (t,))
    assert torch.equal(out, m(x, e, w)) and (tangent - want).abs().max() <= size
    with torch.autograd.forward_ad.dual_level():
        dual = m(x, e, torch.autograd.forward_ad.make_dual(w, t))
        assert torch.equal(torch.autograd.forward_ad.unpack_dual(dual).tangent, tangent)
    fwd, rev = torch.func.jacfwd(lambda w: m(x, e, w))(w), torch.func.jacrev(lambda w: m(x, e, w))(w)
    assert rev.abs().max() > 0 and torch.all((fwd - rev).abs() <= 8 * U * rev.abs())
    ws = torch.stack([w, t])
    assert torch.equal(torch.vmap(lambda v: m(x, e, v))(ws), torch.stack([m(x, e, w), m(x, e, t)]))


def test_experts_gradient_of_padded_slots_is_zero():
    """Beside a token that is not a number, whose rows come first, and where no slot has an expert."""
    m, n, g = experts_of(22)
    x, w, up = n(9, 64), n(9, 3), n(9, 64)
    e = torch.stack([torch.randperm(6, generator=g, device=DEV)[:3] for _ in range(9)])
    e[0] = torch.tensor([0, 1, 2], device=DEV)
    e[4, 0] = e[4, 2] = e[7, 1] = -1

    def grad(x, e, w):
        v = w.clone().requires_grad_()
        (m(x, e, v)[1:] * up[1:]).sum().backward()
        return v.grad

    want = grad(x, e, w)
    x[0] = NAN
    got = grad(x, e, w)
    assert torch.equal(got[1:], want[1:]) and got[4, 0] == 0 and got[4, 2] == 0 and got[7, 1] == 0
    assert (grad(x, torch.full_like(e, -1), torch.full_like(w, NAN)) == 0).all()


# ------------------------------------------------------------------- route --

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("topk", [61, 62, 63, 64])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_one_group_by_two_is_ordered_by_its_logits(sigmoid, topk, dtype):
    """Scores that no number of bits tells apart (sigmoids of 1, softmax terms of 0), one group valued
    by its two largest, so many experts that a kernel of its own takes them: the logits' order."""
    E = 64
    step = torch.arange(E).float()
    logits = torch.stack([40 + 0.5 * step, 100 - step, -1200 + 4 * step, -900 - 8 * ((step * 37) % E),
                          (step * 29) % E * 16 - 1000])
    logits[3, 5] = 0.0                                   # the others vanish beside it
    logits = logits.to(DT[dtype])
    e, w = lb.lowbit_moe_route(logits.to(DEV), topk, score=lb.ROUTE_SIGMOID if sigmoid else lb.ROUTE_SOFTMAX,
                               groups=1, topk_groups=1, group_best=2)
    assert torch.equal(e.cpu().long(), logits.float().sort(dim=1, descending=True, stable=True).indices[:, :topk])
    ref_e, ref_w = o.route(f64(logits), topk, sigmoid=sigmoid, groups=1, topk_groups=1, best=2)
    assert np.array_equal(e.cpu().numpy(), ref_e)
    # (64-bit weights, rounded once)
    assert np.all(np.abs(f64(w) - ref_w) <= 1.01 * U * ref_w + 2.0 ** -149)
    one = lb.lowbit_moe_route(logits.to(DEV), topk, score=lb.ROUTE_SIGMOID if sigmoid else lb.ROUTE_SOFTMAX)
    assert torch.equal(e, one[0]) and torch.equal(w, one[1])


# -------------------------------------------------------------- group_rows --

# Every schedule: a block an expert with one, four and sixteen waves (the last with one run of steps a
# wave, and several), a block a chunk in one launch, two launches with chunks of 1024 and 4096, three,
# and a sort by each of an id's digits.
ORDERS = [(3, 5, 4), (700, 3, 60), (1025, 7, 5), (2049, 8, 256), (5001, 4, 900), (5001, 4, 1500), (8192, 8, 61),
          (8193, 1, 65536), (65535, 1, 901), (16385, 4, 3000), (12001, 8, 256), (70000, 2, 33), (70000, 2, 901),
          (40000, 3, 900), (70001, 8, 257), (700000, 6, 61), (524289, 8, 3), (513, 1, 65536), (600, 1, 65535), (1024, 1, 65536),
          (9000, 4, 1024), (40001, 1, 901), (11000, 7, 512 * 9), (16385, 8, 512 * 9 + 1), (60000, 3, 2047), (33000, 1, 5000)]


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("T, k, E", ORDERS)
def test_group_rows_of_every_schedule_is_the_stable_order(T, k, E, kind):
    """Against a stable sort on the CPU: ids spread out, all alike, and of the first and last only; without
    a workspace and with one, whose end is kept."""
    g = torch.Generator().manual_seed(T + E)
    for ids in (torch.randint(-1, E + 1, (T, k), generator=g), torch.full((T, k), E // 2),
                torch.randint(0, 2, (T, k), generator=g) * (E - 1)):
        dev = ids.to(kind).to(DEV)
        need = lb.load().lowbit_group_rows_workspace_bytes(T, k, E)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
        got = lb.lowbit_group_rows(dev, E, workspace=ws[:need] if need else None)
        if need:
            assert all(torch.equal(a, b) for a, b in zip(got, lb.lowbit_group_rows(dev, E)))
            if T * k * E <= 1 << 30:
                assert all(torch.equal(a, b) for a, b in zip(got, lb.lowbit_group_rows(dev, E, workspace=ws[:need - 1])))
            assert (ws[need:] == 255).all()
        rows, offsets, position = (v.cpu().long() for v in got)
        key = torch.where((ids >= 0) & (ids < E), ids, E).view(-1)
        order = torch.argsort(key, stable=True)
        place = torch.empty_like(order)
        place[order] = torch.arange(T * k)
        assert torch.equal(rows, order // k)
        assert offsets[0] == 0 and torch.equal(offsets[1:], torch.bincount(key, minlength=E + 1)[:E].cumsum(0))
        assert torch.equal(position.view(-1), torch.where(key < E, place, -1))


# ----------------------------------------------------------------- the sum --

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T, N", [(1, 16), (1, 2048), (3, 5008), (64, 272), (300, 1024), (2000, 64)])
def test_combine_is_torch_s_sum_up_to_31_slots(T, N, dtype):
    """Bit for bit: products in fp32, their sum over the slots by torch, rounded once, as F8Experts
    computes it where a derivative may be asked for."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T + N)
    for k in range(1, 32):
        y = torch.randn(T * k, N, generator=g, device=DEV).to(DT[dtype])
        w = torch.rand(T, k, generator=g, device=DEV) - 0.25
        position = torch.randperm(T * k, generator=g, device=DEV).view(T, k).int()
        position = torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.1, -1, position)
        terms = y[position.clamp(min=0).long()].float() * w.unsqueeze(-1)
        want = torch.where((position >= 0).unsqueeze(-1), terms, 0.0).sum(1).to(DT[dtype])
        assert torch.equal(lb.lowbit_moe_combine(y, position, w), want), k


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("k", [1, 8, 16, 31, 32, 47, 64])
def test_experts_sum_is_one_with_and_without_a_derivative(k, dtype):
    """Bit for bit, and that of torch over the slots' rows."""
    m, n, g = experts_of(23, E=64, H=272, I=48, dtype=DT[dtype])
    x, w = n(50, 272).to(DT[dtype]), torch.rand(50, k, generator=g, device=DEV)
    e = torch.stack([torch.randperm(64, generator=g, device=DEV)[:k] for _ in range(50)])
    e = torch.where(torch.rand(50, k, generator=g, device=DEV) < 0.1, -1, e)
    out = m(x, e, w)
    assert torch.equal(m(x, e, w.clone().requires_grad_()), out)
    assert torch.equal(torch.func.jvp(lambda v: m(x, e, v), (w,), (w,))[0], out)
    # the slots' rows by the same calls (a linear by expert of fewer rows may add in another order)
    op = torch.ops.lowbit
    xq, xs = op.quantize_act_f8(x)
    rows, offsets, position = op.group_rows(e, 64)
    gate, up = op.linear_f8_grouped(xq, xs, rows, offsets, m.gate_up, m.gate_up_scale, None, m.dtype).split(48, dim=-1)
    aq, a_s = op.quantize_act_f8(torch.nn.functional.silu(gate) * up)
    slots = op.linear_f8_grouped(aq, a_s, None, offsets, m.down, m.down_scale, None, m.dtype)
    terms = slots[position.clamp(min=0).long()].float() * w.unsqueeze(-1)
    assert torch.equal(torch.where((position >= 0).unsqueeze(-1), terms, 0.0).sum(1).to(DT[dtype]), out)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("spread", [0.01, 1.5, 20.0])
@pytest.mark.parametrize("E, k", [(1, 1), (8, 2), (60, 4), (64, 8), (130, 7), (256, 8), (257, 8), (512, 10), (1023, 9), (1024, 64)])
def test_route_softmax_weights_as_they_are(E, k, spread, dtype):
    """Weights divided by the sum over all experts: each term of it is good to 2^-32 of itself, so a weight
    is off by its own rounding to fp32 and 1 % of that for all else."""
    for T in (1, 33, 2100):
        g = torch.Generator(device=DEV)
        g.manual_seed(E + T)
        logits = (spread * torch.randn(T, E, generator=g, device=DEV)).to(DT[dtype])
        logits[T // 2] = logits[T // 2].abs().neg() * 40      # a row far from 0, with terms that vanish
        if E > 4:
            logits[0, ::3], logits[T - 1, 1::2] = NEG, torch.finfo(DT[dtype]).min
        e, w = lb.lowbit_moe_route(logits, k, renormalize=False, scale=0.75)
        want = 0.75 * torch.softmax(logits.double(), 1).gather(1, e.long().clamp(min=0))
        want = torch.where(e >= 0, want, 0.0)
        assert torch.all((w.double() - want).abs() <= 1.01 * U * want + 2.0 ** -149)
    e, w = lb.lowbit_moe_route(torch.full((3, E), NEG, device=DEV, dtype=DT[dtype]), k, renormalize=False)
    assert (e == -1).all() and (w == 0).all()


def test_group_rows_by_digits_in_a_graph_and_without_positions():
    """Replays with new ids, eager calls between them, each with its own workspace; ids far outside."""
    T, k, E = 9000, 4, 5000
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    ids = torch.randint(-3, E + 3, (T, k), generator=g, device=DEV)
    ids[5] = torch.tensor([2 ** 40 + 1, -2 ** 63, 2 ** 63 - 1, 2 ** 31], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lb.lowbit_group_rows(ids, E)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lb.lowbit_group_rows(ids, E)
    for i in range(4):
        ids[:] = torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.5, ids, torch.randint(-3, E + 3, (T, k), generator=g, device=DEV))
        graph.replay()
        want = lb.lowbit_group_rows(ids, E)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        key = torch.where((ids >= 0) & (ids < E), ids, E).view(-1)
        assert torch.equal(got[0].long(), torch.argsort(key, stable=True) // k)
