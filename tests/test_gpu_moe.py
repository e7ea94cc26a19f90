"""The operators around the experts on the GPU against the 64-bit oracle: routing, grouping of rows,
the experts' sum, and the run of them with the linears by expert.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
  * route: experts are equal.  Weights are computed in 64 bits from the logits and rounded once: u of
    themselves, taken as 1.01 u for the 64-bit steps (scale is the call's, an fp32 number).  Softmax
    without renormalization, without a bias, divides by a sum of fp32 exps: an exp of x = l - top is
    off by x's rounding, u |x| e^x <= 0.37 u, and by its own, 2 u (a unit in the last place); up to
    32 values of a lane and 6 steps over the lanes add 38 u: 42 u with the rounding of the result;
  * combine: k products and k (+ 1) additions in fp32: (2 k + 1) u of the terms' magnitudes' sum,
    and half a step of the output type.
"""
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


def half_step(y, dtype):
    eps = torch.finfo(dtype).eps
    return np.maximum(np.abs(y), float(torch.finfo(dtype).tiny)) * (eps / 2)


# ------------------------------------------------------------------- route --

def check_route(logits, k, bias=None, sigmoid=False, groups=1, topk_groups=1, best=1, renormalize=True, scale=1.0):
    got = lb.lowbit_moe_route(logits.to(DEV), k, bias=None if bias is None else bias.to(DEV),
                              score=lb.ROUTE_SIGMOID if sigmoid else lb.ROUTE_SOFTMAX, groups=groups,
                              topk_groups=topk_groups, group_best=best, renormalize=renormalize, scale=scale)
    e, w = o.route(f64(logits), k, bias=None if bias is None else f64(bias), sigmoid=sigmoid, groups=groups,
                   topk_groups=topk_groups, best=best, renormalize=renormalize, scale=float(np.float32(scale)))
    assert got[0].dtype == torch.int32 and got[1].dtype == torch.float32
    assert np.array_equal(got[0].cpu().numpy(), e)
    g = f64(got[1])
    assert np.array_equal(np.isnan(g), np.isnan(w))
    ok = ~np.isnan(w)
    tol = (42 if not sigmoid and not renormalize and bias is None else 1.01) * U
    assert np.all(np.abs(g - w)[ok] <= tol * np.abs(w[ok]) + 2.0 ** -149)
    return got


SHAPES = [(1, 1, 1, 1), (8, 2, 1, 1), (60, 4, 1, 1), (60, 6, 4, 2), (64, 8, 1, 1), (65, 8, 1, 1), (128, 6, 16, 3),
          (130, 7, 13, 5), (160, 6, 8, 3), (256, 8, 8, 4), (257, 8, 1, 1), (384, 12, 3, 2), (320, 64, 64, 20),
          (512, 10, 1, 1), (1023, 9, 33, 7), (1024, 16, 1, 1), (1024, 64, 64, 64), (6, 6, 6, 2), (16, 16, 16, 16)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "softmax+bias", "sigmoid+bias"])
@pytest.mark.parametrize("E, k, groups, topk_groups", SHAPES)
def test_route(E, k, groups, topk_groups, score):
    """Every layout of lanes and groups, each type, weights renormalized and as they are."""
    g = torch.Generator().manual_seed(E * 131 + k)
    for i, (dtype, T) in enumerate([("f32", 37), ("bf16", 5), ("f16", 70)]):
        logits = (2 * torch.randn(T, E, generator=g)).to(DT[dtype])
        bias = 0.2 * torch.randn(E, generator=g) if "bias" in score else None
        check_route(logits, k, bias=bias, sigmoid="sigmoid" in score, groups=groups, topk_groups=topk_groups,
                    best=2 if bias is not None and i != 1 else 1, renormalize=i != 2, scale=(1.0, 2.5, 0.3)[i])


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 1000, 4097])
def test_route_rows(T):
    g = torch.Generator().manual_seed(T)
    check_route(torch.randn(T, 60, generator=g), 4)
    check_route(torch.randn(T, 300, generator=g).bfloat16(), 5, sigmoid=True, bias=torch.randn(300, generator=g),
                groups=10, topk_groups=3, best=2)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_equal_values_take_the_lowest_index(sigmoid, with_bias):
    E = 96
    bias = torch.full((E,), 0.25) if with_bias else None
    logits = torch.zeros(6, E)
    logits[1] = torch.arange(E) % 3                      # 32 of each value
    logits[2, 50:] = 1.0
    logits[3] = -0.0
    logits[3, ::2] = 0.0
    logits[4] = torch.arange(E, 0, -1)
    logits[5] = torch.arange(E)
    for k in (1, 5, 40):
        check_route(logits, k, bias=bias, sigmoid=sigmoid)
    check_route(logits[:4], 6, bias=bias, sigmoid=sigmoid, groups=8, topk_groups=3, best=2 if with_bias else 1)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_neighbours_below_fp32(sigmoid, with_bias):
    """Scores that fp32 cannot tell apart: their order is that of the 64-bit values."""
    E, T = 128, 64
    g = torch.Generator().manual_seed(3)
    base = torch.nextafter(torch.full((T, 1), 0.7), torch.tensor(1.0))
    steps = torch.randint(0, 3, (T, E), generator=g)
    logits = base.expand(T, E).clone()
    for _ in range(2):
        logits = torch.where(steps > 0, torch.nextafter(logits, torch.tensor(9.0)), logits)
        steps = steps - 1
    bias = None
    if with_bias:
        bias = torch.where(torch.rand(E, generator=g) < 0.5, 0.5, float(np.nextafter(np.float32(0.5), np.float32(1))))
    check_route(logits, 7, bias=bias, sigmoid=sigmoid)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("E, groups, topk_groups", [(64, 4, 2), (256, 8, 4), (320, 5, 1), (512, 32, 9)])
def test_route_neighbouring_groups_and_rows_of_one_value(E, groups, topk_groups, with_bias):
    """Groups whose values fp32 cannot tell apart, and rows full of experts that it cannot."""
    g = torch.Generator().manual_seed(E)
    up = lambda t: torch.nextafter(t, torch.tensor(9.0))
    for T in (6, 5000):                                  # both layouts of lanes
        logits = torch.full((T, E), 0.4)
        for _ in range(2):
            logits = torch.where(torch.rand(T, E, generator=g) < 0.3, up(logits), logits)
        logits[T // 2:] = 0.4                            # all alike
        far = torch.randn(T, E, generator=g) - 3         # ... or only the largest of each group
        far.view(T, groups, -1)[:, :, 1] = logits[:, :groups]
        far.view(T, groups, -1)[:, :, 3] = logits[:, groups:2 * groups]
        bias = None
        if with_bias:
            bias = torch.where(torch.rand(E, generator=g) < 0.5, 0.25, float(np.nextafter(np.float32(0.25), np.float32(1))))
        rows = torch.arange(0, T, max(T // 40, 1))
        for l in (logits, far):
            got = lb.lowbit_moe_route(l.to(DEV), 6, bias=None if bias is None else bias.to(DEV), score=lb.ROUTE_SIGMOID,
                                      groups=groups, topk_groups=topk_groups, group_best=2)
            e, _ = o.route(f64(l[rows]), 6, bias=None if bias is None else f64(bias), sigmoid=True, groups=groups,
                           topk_groups=topk_groups, best=2)
            assert np.array_equal(got[0][rows.to(DEV)].cpu().numpy(), e)


@pytest.mark.parametrize("kind", ["f32", "bias", "groups"])
def test_route_many_rows(kind):
    """Some ten million scores: every choice that of 64 bits."""
    T, E, k = 40000, 256, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(17)
    logits = 1.5 * torch.randn(T, E, generator=g, device=DEV)
    kw, c = {}, logits.double()
    if kind != "f32":
        bias = 0.1 * torch.randn(E, generator=g, device=DEV)
        kw, c = dict(bias=bias, score=lb.ROUTE_SIGMOID), torch.sigmoid(c) + bias.double()
    if kind == "groups":
        kw.update(groups=8, topk_groups=4, group_best=2)
        value = c.view(T, 8, 32).topk(2, 2).values.sum(2)
        keep = torch.zeros(T, 8, dtype=torch.bool, device=DEV).scatter_(1, value.topk(4, 1).indices, True)
        c = torch.where(keep.repeat_interleave(32, 1), c, NEG)
    want = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(lb.lowbit_moe_route(logits, k, **kw)[0].long(), want)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups, topk_groups, best", [(1, 1, 1), (6, 2, 1), (6, 2, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_masks(sigmoid, groups, topk_groups, best, with_bias):
    """-inf masks: rows with fewer experts left than k, with one, with none; masked by the bias."""
    E, k = 60, 5
    g = torch.Generator().manual_seed(9)
    logits = torch.randn(12, E, generator=g)
    bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
    if with_bias:
        bias[7], bias[31] = NEG, NEG
    logits[0] = NEG
    logits[1] = NEG
    logits[1, 41] = -3.0
    logits[2, 4:] = NEG
    logits[3, :-4] = NEG
    logits[4, ::2] = NEG
    logits[5] = torch.where(torch.rand(E, generator=g) < 0.95, torch.tensor(NEG), logits[5])
    logits[6, 10:50] = NEG                               # whole groups
    logits[7] = torch.finfo(torch.float32).min           # the type's lowest value is a number, not a mask
    logits[8, 1:] = torch.finfo(torch.float32).min
    logits[9, :3] = torch.finfo(torch.float32).max if sigmoid else 80.0
    for renormalize in (True, False):
        if not sigmoid or renormalize:
            check_route(logits, k, bias=bias, sigmoid=sigmoid, groups=groups, topk_groups=topk_groups, best=best,
                        renormalize=renormalize)


def test_route_not_a_number():
    E, k = 70, 4
    g = torch.Generator().manual_seed(10)
    for bias in (None, torch.randn(E, generator=g)):
        for sigmoid in (False, True):
            logits = torch.randn(9, E, generator=g)
            logits[1, 0], logits[3, 69], logits[4, 33] = NAN, NAN, INF
            logits[5] = NAN
            logits[6], logits[6, 8] = NEG, NAN
            check_route(logits, k, bias=bias, sigmoid=sigmoid)
            check_route(logits, k, bias=bias, sigmoid=sigmoid, groups=10, topk_groups=2)
    bias = torch.zeros(E)
    bias[5], bias[6] = INF, INF                          # always chosen
    logits = torch.randn(3, E, generator=g)
    logits[1, 5] = NEG                                   # but not where it is masked
    check_route(logits, k, bias=bias)
    bias[60] = NAN
    logits[2, 60] = NEG
    check_route(logits, k, bias=bias, sigmoid=True)


def test_route_far_logits():
    """Weights whose scores leave fp32, or 64 bits: the ratios stay."""
    logits = torch.tensor([[-100.0, -101.0, -200.0, -102.0], [-3e4, -3e4 - 1, -3e4 - 2, -3e4 - 3],
                           [500.0, 499.0, -500.0, 0.0], [-1000.0, -1001.0, 700.0, -999.0]])
    for sigmoid in (False, True):
        check_route(logits, 2, sigmoid=sigmoid)
        check_route(logits, 4, sigmoid=sigmoid)
        check_route(logits[:1], 3, sigmoid=sigmoid, bias=torch.tensor([0.0, 1.0, 2.0, 3.0]))


def test_route_same_row_anywhere():
    """A row's answer hangs neither on its place nor on the rows beside it."""
    g = torch.Generator().manual_seed(12)
    row = torch.randn(1, 160, generator=g)
    many = torch.randn(333, 160, generator=g)
    many[::7] = row
    for kw in (dict(), dict(bias=torch.randn(160, generator=g).to(DEV), groups=8, topk_groups=3, group_best=2,
                            score=lb.ROUTE_SIGMOID)):
        e1, w1 = lb.lowbit_moe_route(row.to(DEV), 6, **kw)
        e, w = lb.lowbit_moe_route(many.to(DEV), 6, **kw)
        assert (e[::7] == e1).all() and (w[::7] == w1).all()


def test_route_no_rows_given_outputs_and_neighbours():
    e, w = lb.lowbit_moe_route(torch.empty(0, 8, device=DEV), 2)
    assert e.shape == (0, 2) and w.shape == (0, 2)
    logits = torch.randn(5, 40, device=DEV)
    big_e = torch.full((7, 3), 77, dtype=torch.int32, device=DEV)
    big_w = torch.full((7, 3), 7.0, device=DEV)
    lb.lowbit_moe_route(logits, 3, experts=big_e[1:6], weights=big_w[1:6])
    want = lb.lowbit_moe_route(logits, 3)
    assert torch.equal(big_e[1:6], want[0]) and torch.equal(big_w[1:6], want[1])
    assert (big_e[[0, 6]] == 77).all() and (big_w[[0, 6]] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_logits_off_alignment(dtype):
    """Logits that start at any element, as a slice of a larger buffer does."""
    g = torch.Generator().manual_seed(13)
    flat = torch.randn(1 + 9 * 64, generator=g).to(DT[dtype]).to(DEV)
    for off in (0, 1):
        logits = flat[off:off + 9 * 64].view(9, 64)
        e, w = lb.lowbit_moe_route(logits, 6)
        want = o.route(f64(logits), 6)
        assert np.array_equal(e.cpu().numpy(), want[0])


# -------------------------------------------------------------- group_rows --

def check_group(ids, E):
    got = lb.lowbit_group_rows(ids.to(DEV), E)
    for g, want in zip(got, o.group_rows(ids.numpy(), E)):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), want)
    return got


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
@pytest.mark.parametrize("T, k, E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (64, 1, 3), (65, 1, 300), (100, 7, 16),
                                     (128, 8, 64), (129, 8, 33), (1000, 3, 256), (2049, 8, 10), (5000, 6, 60)])
def test_group_rows(T, k, E, kind):
    g = torch.Generator().manual_seed(T + k + E)
    ids = torch.randint(0, E, (T, k), generator=g).to(kind)
    check_group(ids, E)
    out = torch.rand(T, k, generator=g)
    check_group(torch.where(out < 0.2, -1, torch.where(out < 0.3, E, ids)).to(kind), E)


@pytest.mark.parametrize("T", [1, 70, 3000])
def test_group_rows_edges(T):
    """All to one expert, none to any, the first or the last only, ids far outside."""
    E, k = 9, 2
    for v in (0, 4, E - 1, E, -1, 2 ** 31 - 1, -2 ** 31):
        check_group(torch.full((T, k), v, dtype=torch.int32), E)
    for v in (2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1):       # (not expert 1)
        check_group(torch.full((T, k), v, dtype=torch.int64), E)


def test_group_rows_of_many_experts():
    g = torch.Generator().manual_seed(1)
    check_group(torch.randint(-1, 1 << 16, (40, 3), generator=g), 1 << 16)
    check_group(torch.randint(0, 5000, (700, 2), generator=g), 5000)


@pytest.mark.parametrize("T, k, E", [(3, 5, 4), (700, 3, 60), (1025, 7, 5), (2049, 8, 256), (5001, 4, 900), (5001, 4, 1500),
                                     (8192, 8, 61), (12001, 8, 256), (70000, 2, 33), (40000, 3, 900)])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_group_rows_with_and_without_workspace(T, k, E, kind):
    """Both schedules: the same rows, also where all tokens go one way; the workspace's end kept."""
    g = torch.Generator().manual_seed(T)
    for ids in (torch.randint(-1, E + 1, (T, k), generator=g), torch.full((T, k), E // 2),
                torch.randint(0, 2, (T, k), generator=g) * (E - 1)):
        ids = ids.to(kind).to(DEV)
        need = lb.load().lowbit_group_rows_workspace_bytes(T, k, E)
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
        a = lb.lowbit_group_rows(ids, E)
        b = lb.lowbit_group_rows(ids, E, workspace=ws[:need] if need else None)
        c = lb.lowbit_group_rows(ids, E, workspace=ws[:0] if need else None)      # too small: one launch
        for x, y, z in zip(a, b, c):
            assert torch.equal(x, y) and torch.equal(x, z)
        assert (ws[need:] == 255).all()


def test_group_rows_none():
    rows, offsets, position = lb.lowbit_group_rows(torch.empty(0, 4, dtype=torch.int32, device=DEV), 7,
                                                   offsets=torch.full((8,), 9, dtype=torch.int32, device=DEV))
    assert rows.shape == (0,) and position.shape == (0, 4) and (offsets == 0).all()


def test_group_rows_large():
    """More slots than a prompt has, against a library sort."""
    T, k, E = 70001, 8, 384
    ids = torch.randint(-2, E + 2, (T, k), device=DEV)
    rows, offsets, position = lb.lowbit_group_rows(ids, E)
    key = torch.where((ids >= 0) & (ids < E), ids, E).view(-1)
    order = torch.argsort(key, stable=True)
    assert torch.equal(rows.long(), order // k)
    assert torch.equal(offsets[1:].long(), torch.bincount(key, minlength=E + 1)[:E].cumsum(0))
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=DEV)
    assert torch.equal(position.view(-1).long(), torch.where(key < E, place, -1))


# ----------------------------------------------------------------- combine --

def check_combine(y, position, weights, residual=None, **kw):
    out = lb.lowbit_moe_combine(y.to(DEV), position.to(DEV), weights.to(DEV),
                                residual=None if residual is None else residual.to(DEV), **kw)
    ref, A = o.combine(f64(y), position.numpy(), weights.numpy(), None if residual is None else f64(residual))
    got = f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    tol = (2 * position.shape[1] + 1) * U * A + half_step(ref, y.dtype)
    assert np.all(np.abs(got - ref)[ok] <= tol[ok] * 1.0001)
    return out


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T, k, N", [(1, 1, 1), (1, 8, 2048), (5, 2, 7), (3, 4, 2056), (17, 3, 129), (40, 6, 264),
                                     (2, 13, 5001)])
def test_combine(T, k, N, dtype):
    g = torch.Generator().manual_seed(T * 7 + N)
    y = torch.randn(T * k, N, generator=g).to(DT[dtype])
    position = torch.randperm(T * k, generator=g).view(T, k).to(torch.int32)
    w = torch.rand(T, k, generator=g) - 0.3
    residual = torch.randn(T, N, generator=g).to(DT[dtype])
    check_combine(y, position, w)
    check_combine(y, position, w, residual)
    check_combine(y, torch.where(torch.rand(T, k, generator=g) < 0.4, -1, position).to(torch.int32), w, residual)


def test_combine_slots_without_an_expert():
    """They add nothing, whatever their weight and whatever the rows hold; a position behind the
    rows makes its row NaN; the same position twice counts twice."""
    g = torch.Generator().manual_seed(2)
    y = torch.randn(6, 40, generator=g).bfloat16()
    y[5] = NAN
    w = torch.rand(5, 3, generator=g)
    w[0, 1], w[3, 0] = NAN, INF
    position = torch.tensor([[0, -1, 1], [-1, -1, -1], [2, 2, 3], [-7, 4, -2 ** 31], [0, 6, 1]], dtype=torch.int32)
    out = check_combine(y, position, w)
    assert (out[1] == 0).all() and torch.isnan(out[4]).all()
    out = check_combine(y, position, w, torch.randn(5, 40, generator=g).bfloat16())
    assert torch.isnan(out[4]).all()
    out = lb.lowbit_moe_combine(torch.empty(0, 40, device=DEV), torch.full((2, 3), -1, dtype=torch.int32, device=DEV),
                                torch.ones(2, 3, device=DEV))
    assert (out == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [48, 50])
def test_combine_in_place_and_off_alignment(dtype, N):
    g = torch.Generator().manual_seed(4)
    T, k = 9, 2
    y = torch.randn(T * k, N, generator=g).to(DT[dtype])
    position = torch.randperm(T * k, generator=g).view(T, k).to(torch.int32)
    w = torch.rand(T, k, generator=g)
    residual = torch.randn(T, N, generator=g).to(DT[dtype])
    want = check_combine(y, position, w, residual)
    own = residual.to(DEV)
    assert lb.lowbit_moe_combine(y.to(DEV), position.to(DEV), w.to(DEV), residual=own, out=own) is own
    assert torch.equal(own, want)
    flat = torch.full(((T + 2) * N + 1,), 3.0, dtype=DT[dtype], device=DEV)
    out = flat[1 + N:1 + N + T * N].view(T, N)           # one element off, neighbours kept
    lb.lowbit_moe_combine(y.to(DEV), position.to(DEV), w.to(DEV), residual=residual.to(DEV), out=out)
    assert torch.equal(out, want) and (flat[:1 + N] == 3).all() and (flat[1 + N + T * N:] == 3).all()


def test_combine_rows_past_4_gib():
    """Rows of y whose offsets pass 32 bits, elements and bytes."""
    N, R = 8192, (1 << 32) // 8192 + 40
    y = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
    y[0], y[R - 1], y[R // 2 + 3] = 1.0, 2.0, 4.0
    position = torch.tensor([[0, R - 1], [R // 2 + 3, -1], [R - 2, R]], dtype=torch.int32, device=DEV)
    out = lb.lowbit_moe_combine(y, position, torch.ones(3, 2, device=DEV))
    assert (out[0] == 3).all() and (out[1] == 4).all() and torch.isnan(out[2]).all()


def test_combine_more_rows_than_a_launch_has_blocks():
    T, N, R = (1 << 24) + 70, 1032, 50                   # (a block a row at this width, 34 GB of sums)
    y = torch.randn(R, N, device=DEV).bfloat16()
    at = torch.arange(T, device=DEV)
    position, w = (at % R).int().unsqueeze(1), ((at % 7) / 8).unsqueeze(1)
    residual = torch.zeros(1, N, dtype=torch.bfloat16, device=DEV).expand(T, N).contiguous()
    residual[-1] = 64.0
    out = lb.lowbit_moe_combine(y, position, w, residual=residual, out=residual)
    for t in (*range(0, T - (1 << 20), 1 << 20), (1 << 24) - (1 << 19)):
        s = slice(t, min(t + (1 << 20), T))
        want = y[position[s, 0].long()].float() * w[s]   # (w has three bits: the product is exact)
        if s.stop == T:
            want[-1] += 64.0
        assert torch.equal(out[s], want.bfloat16())


# ------------------------------------------------------- the run together --

def moe_calls(t):
    """Router, grouping, both linears by expert and the sum, on given outputs."""
    lb.lowbit_moe_route(t["logits"], t["k"], bias=t["bias"], score=lb.ROUTE_SIGMOID, groups=4, topk_groups=2,
                        group_best=2, scale=2.0, experts=t["experts"], weights=t["weights"])
    lb.lowbit_group_rows(t["experts"], t["E"], t["rows"], t["offsets"], t["position"])
    lb.lowbit_quantize_act_f8(t["x"], t["xq"], t["xs"])
    lb.lowbit_linear_f8_grouped(t["xq"], t["xs"], t["offsets"], t["w"], t["ws"], None, torch.bfloat16,
                                rows=t["rows"], y=t["y"])
    lb.lowbit_moe_combine(t["y"], t["position"], t["weights"], residual=t["x"], out=t["out"])


def moe_tensors(seed, T, E=16, k=4, H=272):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def n(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    w, ws = lb.lowbit_quantize_weight_f8(n(E, H, H) * 0.06)
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(E=E, k=k, logits=n(T, E), bias=0.1 * n(E), x=n(T, H).bfloat16(), w=w, ws=ws,
                experts=torch.empty(T, k, **i32), weights=torch.empty(T, k, device=DEV),
                rows=torch.empty(T * k, **i32), offsets=torch.empty(E + 1, **i32),
                position=torch.empty(T, k, **i32), xq=torch.empty(T, H, dtype=torch.float8_e4m3fn, device=DEV),
                xs=torch.empty(T, 3, device=DEV), y=torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV),
                out=torch.empty(T, H, dtype=torch.bfloat16, device=DEV))


@pytest.mark.parametrize("T", [1, 50, 777])
def test_router_experts_sum(T):
    """As a block runs, against the same sums from the dequantized codes."""
    t = moe_tensors(T, T)
    t["logits"][T // 2] = NEG                            # a padded token: it keeps the residual
    moe_calls(t)
    e, w = o.route(f64(t["logits"]), t["k"], bias=f64(t["bias"]), sigmoid=True, groups=4, topk_groups=2, best=2,
                   scale=2.0)
    assert np.array_equal(t["experts"].cpu().numpy(), e)
    x = f64(t["xq"].float()) * np.repeat(f64(t["xs"]), 128, 1)[:, :272]
    wt = f64(t["w"].float()) * np.repeat(np.repeat(f64(t["ws"]), 128, 1), 128, 2)[:, :272, :272]
    ref, A = f64(t["x"]).copy(), np.abs(f64(t["x"]))
    for i in range(T):
        for ex, wi in zip(e[i], w[i]):
            if ex >= 0:
                ref[i] += wi * (wt[ex] @ x[i])
                A[i] += wi * (np.abs(wt[ex]) @ np.abs(x[i]))
    # each expert's row is rounded to bf16 (2^-8 of itself), and so is the sum; the linear's own
    # sums add less than 7 * 2^-13 + 2^-15 of the magnitudes
    bound = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 7 * 2.0 ** -13 + 2.0 ** -15) * A
    assert np.all(np.abs(f64(t["out"]) - ref) <= bound)
    assert torch.equal(t["out"][T // 2], t["x"][T // 2])


def test_graph_replays_equal_eager():
    T = 60
    t = moe_tensors(5, T)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe_calls(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe_calls(t)
    for i in range(5):
        new = moe_tensors(100 + i, T)
        for key in ("logits", "x"):
            t[key].copy_(new[key])
        graph.replay()
        got = {key: t[key].clone() for key in ("experts", "weights", "rows", "offsets", "position", "out")}
        torch.cuda.synchronize()
        for key in got:
            t[key].zero_()
        moe_calls(t)
        for key in got:
            assert torch.equal(got[key], t[key]), key


def test_two_streams_at_once():
    """The same calls on two streams, their own outputs: as one after the other."""
    a, b = moe_tensors(1, 300), moe_tensors(2, 300)
    want = []
    for t in (a, b):
        moe_calls(t)
        torch.cuda.synchronize()
        want.append(t["out"].clone())
        t["out"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for t, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                moe_calls(t)
    torch.cuda.synchronize()
    assert torch.equal(a["out"], want[0]) and torch.equal(b["out"], want[1])


def test_explicit_stream_argument():
    s = torch.cuda.Stream()
    logits = torch.randn(50, 64, device=DEV)
    y = torch.randn(100, 80, device=DEV)
    torch.cuda.synchronize()
    e, w = lb.lowbit_moe_route(logits, 2, stream=s)
    rows, offsets, position = lb.lowbit_group_rows(e, 64, stream=s)
    out = lb.lowbit_moe_combine(y, position, w, stream=s.cuda_stream)
    s.synchronize()
    e2, w2 = lb.lowbit_moe_route(logits, 2)
    assert torch.equal(e, e2) and torch.equal(w, w2)
    assert torch.equal(out, lb.lowbit_moe_combine(y, lb.lowbit_group_rows(e2, 64)[2], w2))


def test_modules_and_ops_match_the_calls():
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    r = lnn.MoeRouter(24, 3, "sigmoid", bias=True, groups=4, topk_groups=2, group_best=2, scale=1.5, device=DEV)
    r.bias.copy_(torch.randn(24, generator=g, device=DEV) * 0.1)
    r.half()
    assert r.bias.dtype == torch.float32
    logits = torch.randn(2, 7, 24, generator=g, device=DEV)
    e, w = r(logits)
    e2, w2 = lb.lowbit_moe_route(logits.view(14, 24), 3, bias=r.bias, score=lb.ROUTE_SIGMOID, groups=4,
                                 topk_groups=2, group_best=2, scale=1.5)
    assert torch.equal(e.view(14, 3), e2) and torch.equal(w.view(14, 3), w2)
    m = lnn.F8Experts(24, 64, 48, device=DEV).set_weight(torch.randn(24, 96, 64, device=DEV) * 0.1,
                                                         torch.randn(24, 64, 48, device=DEV) * 0.1)
    x = torch.randn(2, 7, 64, generator=g, device=DEV).bfloat16()
    out = m(x, e, w)
    assert out.shape == x.shape
    assert torch.equal(out, m(x, e.long(), w.double()))
    assert torch.equal(out, m(x, e.to(torch.uint8), w))
    fn = torch.compile(lambda l, x: m(x, *r(l)), fullgraph=True, backend="aot_eager")
    assert torch.equal(fn(logits, x), out)


def test_experts_keep_the_gradient_of_the_routing_weights():
    """As a router that is trained beside frozen experts needs it.  The sum is linear in the weights:
    its gradient is the product of the output's with each slot's row, 64 products summed in fp32."""
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    m = lnn.F8Experts(6, 64, 48, dtype=torch.float32, device=DEV)
    m.set_weight(torch.randn(6, 96, 64, generator=g, device=DEV) * 0.1, torch.randn(6, 64, 48, generator=g, device=DEV) * 0.1)
    x = torch.randn(11, 64, generator=g, device=DEV)
    e = torch.stack([torch.randperm(6, generator=g, device=DEV)[:3] for _ in range(11)])
    e[2, 1] = e[5, 0] = -1
    w = torch.rand(11, 3, generator=g, device=DEV)
    up = torch.randn(11, 64, generator=g, device=DEV)
    wg = w.clone().requires_grad_()
    out = m(x, e, wg)
    assert torch.equal(out.detach(), m(x, e, w))
    (out * up).sum().backward()
    for j in range(3):
        one = torch.zeros_like(w)
        one[:, j] = 1.0
        terms = (up * m(x, e, one)).double()             # slot j's rows, exactly
        assert torch.all((wg.grad[:, j] - terms.sum(-1)).abs() <= 2 * 65 * U * terms.abs().sum(-1))
    assert wg.grad[2, 1] == 0 and wg.grad[5, 0] == 0


def test_results_carry_no_gradient():
    logits = torch.randn(4, 8, device=DEV, requires_grad=True)
    _, w = lb.lowbit_moe_route(logits, 2)
    assert not w.requires_grad
    with pytest.raises(RuntimeError):
        torch.ops.lowbit.moe_route(logits, None, 2, 0, 1, 1, 1, True, 1.0)[1].sum().backward()
