"""Low-rank adapters on the GPU at the edges of their numbers: infinite elements, x A^T far outside the
call's type; tolerances as in test_gpu_lora.py."""
import numpy as np
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn
from oracle import moe_oracle as o
from tests.test_gpu_lora import DEV, DT, INF, NAN, call, f64, inputs, plan, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lowbit_lib):
    return lowbit_lib


# One launch (ranks to 32, one and two steps of columns) and two, ranks of one pass and of several.
INF_SHAPES = [(1, 1, 8, 16, 40), (40, 20, 16, 272, 300), (60, 30, 32, 144, 1200), (70, 2, 16, 528, 264), (300, 2, 64, 96, 200),
              (90, 2, 136, 80, 136), (33, 2, 256, 64, 150)]


def reference(t):
    with np.errstate(all="ignore"):
        return o.lora(f64(t["x"]), f64(t["a"]), f64(t["b"]), f64(t["scales"]), t["ids"].numpy(), f64(t["base"]))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, L, rank, K, N", INF_SHAPES)
def test_lora_infinite_elements_of_b(M, L, rank, K, N, dtype):
    """One infinite element in every third column: +-inf there by the sign of its t, whatever t's size;
    two of them: +-inf or not a number, as their signs are; the other columns as without any."""
    t = inputs(M + rank, M, L, rank, K, N, dtype, ids=torch.arange(M) % L)
    # x . a over a span of sizes: ranks of one row from 1 down to 2^-30 of its largest
    fade = torch.linspace(0, -30 if dtype != "f16" else -8, rank).round()
    t["a"] = (t["a"].float() * torch.exp2(fade)[None, :, None]).to(DT[dtype])
    want = call(t)
    g = torch.Generator().manual_seed(rank)
    cols = torch.arange(0, N, 3)
    at = torch.randint(0, rank, (len(cols),), generator=g)
    sign = torch.randint(0, 2, (len(cols),), generator=g).float() * 2 - 1
    t["b"] = t["b"].clone()
    t["b"][:, cols, at] = (sign * INF).to(DT[dtype])
    two = cols[1::4]
    t["b"][:, two, (at[1::4] + 1) % rank] = INF
    y = call(t)
    x, a = f64(t["x"]), f64(t["a"])
    ts = np.stack([a[l] @ x[m] for m, l in enumerate(t["ids"].tolist())])           # [M, rank]
    # (no t is so near 0 that its sign is in doubt: sums of K products in fp32)
    size = np.stack([np.abs(a[l]) @ np.abs(x[m]) for m, l in enumerate(t["ids"].tolist())])
    sure = (np.abs(ts) > (2 * (K / 32 + 112) + 1) * 2.0 ** -24 * size).all(1)
    assert sure.mean() > 0.9
    ref = reference(t)[0]
    got = f64(y)
    assert np.isinf(ref[:, cols]).sum() > 0 or M == 1
    assert np.array_equal(np.isnan(got)[sure], np.isnan(ref)[sure])
    assert np.array_equal(np.isposinf(got)[sure], np.isposinf(ref)[sure])
    assert np.array_equal(np.isneginf(got)[sure], np.isneginf(ref)[sure])
    rest = [n for n in range(N) if n % 3]
    assert torch.equal(y[:, rest], want[:, rest])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, L, rank, K, N", INF_SHAPES[1:5])
def test_lora_t_far_below_the_rows_largest_meets_an_infinity(M, L, rank, K, N, dtype):
    """Ranks so small beside the row's largest that a number of the type keeps nothing of them, or
    below the type's smallest number altogether: their sign still decides."""
    t = inputs(M + 1, M, L, rank, K, N, dtype, ids=torch.arange(M) % L)
    x, a = torch.ones(M, K), torch.zeros(L, rank, K)
    x[:, 1:] = 0
    x[1::2, 0] = -1
    a[:, :, 0] = 4.0
    tiny = {"f16": 2.0 ** -24, "bf16": 2.0 ** -120, "f32": 2.0 ** -120}[dtype]
    a[:, 1::2, 0] = tiny
    a[:, 3::4, 0] = -tiny
    t["x"], t["a"] = x.to(DT[dtype]), a.to(DT[dtype])
    t["scales"] = torch.full((L,), {"f16": 2.0 ** -60, "bf16": 2.0 ** -20, "f32": 1.0}[dtype])
    t["b"] = t["b"].clone()
    t["b"][:, 5, 1], t["b"][:, 6, 3], t["b"][:, 7, 0] = INF, INF, -INF
    ref, got = reference(t)[0], f64(call(t))
    for n in (5, 6, 7):
        assert np.isinf(ref[:, n]).all() and np.array_equal(got[:, n], ref[:, n])
    assert np.isfinite(got[:, 8:]).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, L, rank, K, N", INF_SHAPES)
def test_lora_not_finite_adapters_and_rows(M, L, rank, K, N, dtype):
    """Infinities in x and a reach their rows as the definition has them, NaN in b its column, NaN in a
    its adapter's rows; infinite t times an infinite b is infinite."""
    t = inputs(M + 2 * rank, M, L, rank, K, N, dtype, ids=torch.arange(M) % L)
    for k in ("x", "a", "b"):
        t[k] = t[k].clone()
    # (every factor positive: no sum holds two infinities of unlike signs)
    t["x"], t["a"], t["b"] = t["x"].abs() + 0.125, t["a"].abs() + 0.125, t["b"].abs() + 0.125
    plain = call(t)
    t["x"][M // 2, 3] = INF
    t["b"][:, N // 2, rank - 1] = INF
    t["b"][:, N // 3, 0] = NAN
    y = call(t)
    assert (y[M // 2, [n for n in range(N) if n != N // 3]] == INF).all()
    assert (y[:, N // 2] == INF).all() and torch.isnan(y[:, N // 3]).all()
    rows = [m for m in range(M) if m != M // 2]
    cols = [n for n in range(N) if n not in (N // 2, N // 3)]
    assert torch.equal(y[rows][:, cols], plain[rows][:, cols])
    t["a"][0, rank // 2, 1] = NAN
    assert torch.isnan(call(t)[0]).all()


@pytest.mark.parametrize("M", [1, 40])
def test_lora_bf16_largest_t(M):
    """t between bf16's largest number and fp32's: it is finite, and so is its product."""
    rank, K, N = 16, 16, 40
    t = inputs(9, M, 1, rank, K, N, "bf16", ids=torch.zeros(M, dtype=torch.int64))
    x, a = torch.zeros(M, K), torch.zeros(1, rank, K)
    x[:, 0], x[:, 1] = 2.0 ** 64, 2.0 ** 63
    a[:, :, 0], a[:, :, 1] = 1.9921875 * 2.0 ** 63, 1.9921875 * 2.0 ** 56          # t = (2 - 2^-7) (1 + 2^-8) 2^127
    t["x"], t["a"] = x.bfloat16(), a.bfloat16()
    t["scales"] = torch.ones(1)
    t["b"] = torch.zeros(1, N, rank).bfloat16()
    t["b"][0, :, 5] = 2.0 ** -126
    ref, At, Ab, Am = reference(t)
    value = 1.9921875 * (1 + 2.0 ** -8)
    assert torch.finfo(torch.bfloat16).max < value * 2.0 ** 127 < torch.finfo(torch.float32).max
    assert np.all(np.abs(f64(call(t)) - ref) <= tolerance(ref, At, Ab, Am, K, rank, torch.bfloat16))


# (x and a, scale, b): powers of two; t = x A^T times the scale is some 2^(2 xa + 3.5) scale
FAR = {"huge": (11, -4, -23), "largest": (15, -13, -24), "tiny": (-14, -3, 12), "smaller": (-14, -11, 15),
       "scale up": (-14, 14, 8), "scale down": (14, -28, -4)}


@pytest.mark.parametrize("M, L, rank, K, N", [(37, 1, 16, 128, 48), (45, 3, 24, 144, 70), (300, 2, 64, 112, 130)])
@pytest.mark.parametrize("kind", FAR)
def test_lora_f16_t_outside_fp16_and_y_within(kind, M, L, rank, K, N):
    """x A^T (before and behind its scale) beyond fp16's largest number, or below its smallest, with y
    an ordinary number: y is right where the base alone, or zeros, would not be."""
    xa, scale, b = FAR[kind]
    g = torch.Generator().manual_seed(M + len(kind))
    t = inputs(5, M, L, rank, K, N, "f16", ids=torch.arange(M) % L)
    unit = lambda *shape: (torch.rand(*shape, generator=g) + 0.5) * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
    # (up to 2^15 and down to 2^-14 in x and a, 2^-24 in b, where one bit is all there is)
    t["x"], t["a"] = (unit(M, K) * 2.0 ** xa).half(), (unit(L, rank, K) * 2.0 ** xa).half()
    t["b"] = (unit(L, N, rank) * 2.0 ** b).half()
    t["scales"] = torch.full((L,), 2.0 ** scale)
    t["base"] = torch.zeros(M, N).half()
    y, At, Ab, Am = reference(t)
    tol = tolerance(y, At, Ab, Am, K, rank, torch.float16)
    size = np.abs(f64(t["x"]) @ f64(t["a"])[0].T)[np.arange(M) % L == 0] * (1.0 if kind.startswith("scale") else 2.0 ** scale)
    outside = (size > 65504) if kind in ("huge", "largest", "scale down") else (size < 2.0 ** -14)
    fits = np.abs(y) < 60000
    assert outside.mean() > 0.9 and fits.mean() > 0.9 and np.mean(np.abs(y) > 8 * tol) > 0.5
    err = np.abs(f64(call(t)) - y)
    assert np.all(err[fits] <= tol[fits]), f"worst {np.max((err / tol)[fits])}"


@pytest.mark.parametrize("M, N", [(20, 40), (300, 264)])
@pytest.mark.parametrize("with_base", [False, True])
def test_op_lora_keeps_base_in_rows_that_are_not_named(with_base, M, N):
    """Rows that a plan of as many entries, of more or of fewer leaves out: base, or 0; a whole plan
    the same with and without a copy of base."""
    t = inputs(31, M, 2, 16, 48, N, "bf16", ids=torch.arange(M) % 2)
    d = {k: v.to(DEV) for k, v in t.items() if torch.is_tensor(v)}
    base = d["base"] if with_base else None
    want = torch.ops.lowbit.lora(d["x"], d["a"], d["b"], d["scales"], *plan(t), base, True)
    assert torch.equal(torch.ops.lowbit.lora(d["x"], d["a"], d["b"], d["scales"], *plan(t), base), want)
    rest = base if with_base else torch.zeros_like(want)
    kept = d["base"].clone()
    for entries in (M, 2 * M, M - 3):
        named = torch.arange(0, M // 2 * 2, 4)           # (of adapter 0)
        rows = torch.full((entries,), -1)
        rows[:len(named)] = named
        rows[len(named):len(named) + 2] = torch.tensor([M, 2 ** 31 - 1])
        junk = torch.full((M, N), NAN, dtype=torch.bfloat16, device=DEV)       # (memory that is likely taken next)
        del junk
        y = torch.ops.lowbit.lora(d["x"], d["a"], d["b"], d["scales"], rows.int().to(DEV),
                                  torch.tensor([0, entries, entries], dtype=torch.int32, device=DEV), base)
        others = [m for m in range(M) if m not in named.tolist()]
        assert torch.equal(y[named.to(DEV)], want[named.to(DEV)]) and torch.equal(y[others], rest[others])
    assert torch.equal(d["base"], kept)
