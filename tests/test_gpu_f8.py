"""The 8-bit path on the GPU against the 64-bit oracle.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32):
  * linear: the products of two e4m3 numbers are exact in fp32; a block's 128 products are summed
    in fp32 by the matrix core (at most 128 additions, each within 2u of the magnitudes' sum even
    where it truncates), then the two scales' product, its product with the block sum and the sum
    over kb blocks (3 + kb roundings) and the bias: |err| <= (2 * 128 + kb + 5) u A, A the sum of
    the magnitudes, plus half a step of the output type.  With 16-bit outputs the products go
    through the fp8 matrix instruction, which aligns each eight consecutive products to the largest
    and cuts off what is below 2^-13 of it: at most seven of them lose less than 2^-13 of the
    largest each, so the eight's sum loses at most 7 * 2^-13 of its magnitudes, and so does A;
  * norm: the sum of squares of K values, in any order of at most K / 64 + 32 additions in a row,
    halved by the square root, then at most 8 single roundings: relative error of y at most
    d = (K / 128 + 24) u; a code adds half a step: 1/2 scale (int8), 2^-4 |y| or 2^-10 scale (e4m3).
Quantizers without a norm are bitwise equal to the oracle's.
"""
import numpy as np
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn
from oracle import f8_oracle as o
import oracle

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def patterns(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def up8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).view(F8).to(DEV)


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def half_step(y, dtype):
    """Half a step of `dtype` at values y (of its smallest numbers below its normal range)."""
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(y) * fi.eps / 2, fi.smallest_normal * fi.eps / 2)


def close(y, ref, A, kb, dtype, what):
    got = f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    sums = ((2 * 128 + kb + 5) * U + (0 if dtype == torch.float32 else 7 * 2.0 ** -13)) * A
    tol = sums + half_step(np.abs(ref) + sums, dtype)
    # beyond the type's largest number: infinity from half a step above it on
    fi = torch.finfo(dtype)
    over = fi.max * (1 + fi.eps / 4)
    inf = np.isinf(got)
    assert np.all(np.sign(got[inf]) == np.sign(ref[inf])) and np.all(np.abs(ref[inf]) + sums[inf] >= over), what
    assert np.all(inf[np.abs(ref) - sums >= over]), what
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= tol) & ~np.isnan(ref) & ~inf
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.nanmax(np.abs(got - ref) / tol):.3g} of the tolerance"


def random_codes(rng, shape):
    """Any finite e4m3 pattern, small magnitudes as likely as large ones."""
    p = rng.integers(0, 127, shape) | (rng.integers(0, 2, shape) << 7)
    return p.astype(np.uint8)


def scales(rng, shape):
    return np.exp(rng.uniform(-6, 2, shape)).astype(np.float32)


def linear_inputs(seed, M, N, K, dtype, bias, lead=()):
    rng = np.random.default_rng(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    xq, wq = random_codes(rng, (M, K)), random_codes(rng, (*lead, N, K))
    xs, ws = scales(rng, (M, kb)), scales(rng, (*lead, nb, kb))
    b = torch.from_numpy(rng.standard_normal((*lead, N)).astype(np.float32)).to(DT[dtype]) if bias else None
    return xq, xs, wq, ws, b


def run_linear(seed, M, N, K, dtype, bias=False):
    xq, xs, wq, ws, b = linear_inputs(seed, M, N, K, dtype, bias)
    y = lb.lowbit_linear_f8(up8(xq), up(xs), up8(wq), up(ws), None if b is None else b.to(DEV), DT[dtype])
    ref, A = o.linear_f8(xq, xs, wq, ws, None if b is None else f64(b))
    close(y, ref, A, xs.shape[1], DT[dtype], f"M={M} N={N} K={K} {dtype}")
    return y


# ------------------------------------------------------------- quantizers --

def awkward(rng, M, K, dtype):
    x = torch.from_numpy((rng.standard_normal((M, K)) * np.exp(rng.uniform(-20, 20, (M, 1)))).astype(np.float32))
    x = x.clamp(-6e4, 6e4).to(DT[dtype])
    if M >= 6:
        x[0] = 0.0
        x[1, K // 2] = float("nan")
        x[2, K - 1] = float("inf")
        x[3, 0] = -float("inf")
        x[4] = 1e-7 if dtype == "f16" else 1e-36
        x[5] = torch.arange(K).remainder(40).sub(20).to(DT[dtype])
    return x


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, K", [(1, 16), (7, 128), (9, 144), (6, 2080), (33, 4096), (8, 14336)])
def test_quantize_act_f8_is_bit_exact(dtype, M, K):
    x = awkward(np.random.default_rng(M * K), M, K, dtype)
    q, s = lb.lowbit_quantize_act_f8(x.to(DEV))
    rq, rs = o.quantize_f8_rows(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(patterns(q), rq)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 16), (128, 128), (130, 144), (3, 200, 272), (300, 2064)])
def test_quantize_weight_f8_is_bit_exact(dtype, shape):
    rng = np.random.default_rng(sum(shape))
    w = torch.from_numpy((rng.standard_normal(shape) * 0.02).astype(np.float32)).to(DT[dtype])
    w2 = w.view(-1, shape[-1])
    w2[0, -1] = float("nan") if shape[0] == 300 else 3.0
    q, s = lb.lowbit_quantize_weight_f8(w.to(DEV))
    for e, m in enumerate(w.view(-1, *shape[-2:])):
        rq, rs = o.quantize_f8_weight(m.float().numpy())
        assert np.array_equal(s.view(-1, *s.shape[-2:])[e].cpu().numpy(), rs, equal_nan=True)
        assert np.array_equal(patterns(q.view(-1, *shape[-2:])[e]), rq)


# ------------------------------------------------------------------- norm --

def check_norm(x, r, g, eps, fmt, q, s, h, y, dtype):
    K = x.shape[1]
    if r is None:
        hh = x
    else:
        hh = (x.float() + r.float()).to(DT[dtype])
        assert torch.equal(h.cpu().nan_to_num(7.0), hh.nan_to_num(7.0))
        assert torch.equal(h.cpu().isnan(), hh.isnan())
    ref = o.rmsnorm(f64(hh), None if g is None else f64(g), eps)
    d = (K / 128 + 24) * U
    if y is not None:
        got = f64(y)
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        tol = d * np.abs(ref) + half_step(ref * (1 + d), DT[dtype]) + 2.0 ** -149
        with np.errstate(invalid="ignore"):
            assert not (~(np.abs(got - ref) <= tol) & ~np.isnan(ref) & ~np.isinf(got)).any()
    if fmt == lb.Q8_NONE:
        return
    M = x.shape[0]
    span = K if fmt == lb.Q8_I8 else 128
    top = 127.0 if fmt == lb.Q8_I8 else 448.0
    s = f64(s).reshape(M, -1)
    codes = q.cpu().numpy().astype(np.float64) if fmt == lb.Q8_I8 else o.E4M3[patterns(q)]
    for b in range(s.shape[1]):
        v, c = ref[:, b * span:(b + 1) * span], codes[:, b * span:(b + 1) * span]
        bad = np.isnan(v).any(1)
        assert np.array_equal(np.isnan(s[:, b]), bad)
        assert np.all(c[bad] == 0)
        v, c, sb = v[~bad], c[~bad], s[~bad, b]
        amax = np.abs(v).max(1)
        zero = amax < 2.0 ** -110
        assert np.all(sb[zero] == 0) and np.all(c[zero] == 0)
        v, c, sb, amax = v[~zero], c[~zero], sb[~zero], amax[~zero]
        assert np.all(np.abs(sb - amax / top) <= (d + 2 * U) * amax / top)
        full = sb[:, None]
        step = 0.5 * full if fmt == lb.Q8_I8 else np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * full)
        assert np.all(np.abs(c * full - v) <= step * (1 + 2 * d) + 2 * d * np.abs(v))
        assert np.all(np.abs(c).max(1) == top)       # the largest value takes the largest code


NORM_K = [16, 32, 128, 160, 512, 544, 1024, 1040, 2048, 2080, 2560, 2576, 4096, 4112, 8192, 8224, 14336, 16384, 16416,
          32768, 32800, 40960]


@pytest.mark.parametrize("fmt", [lb.Q8_NONE, lb.Q8_I8, lb.Q8_F8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", NORM_K)
def test_norm(dtype, fmt, K):
    if fmt == lb.Q8_I8 and K % 32:
        K += 16
    for M, res, gain, want_y in [(1, True, True, True), (7, False, True, False), (5, True, False, False)]:
        if fmt == lb.Q8_NONE:
            want_y = True
        rng = np.random.default_rng(K + M)
        mk = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[dtype])  # noqa: E731
        x, r, g = mk(M, K) * 3, mk(M, K) if res else None, mk(K) if gain else None
        on = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        q, s, h, y = lb.lowbit_add_rmsnorm_q8(on(x), on(g), 1e-5, fmt, residual=on(r), want_y=want_y)
        assert (y is not None) == want_y and (h is not None) == res and (q is None) == (fmt == lb.Q8_NONE)
        check_norm(x, r, g, float(np.float32(1e-5)), fmt, q, s, h, y, dtype)


@pytest.mark.parametrize("fmt", [lb.Q8_I8, lb.Q8_F8])
@pytest.mark.parametrize("K", [96, 1056, 2528, 4096, 20512, 33024])
def test_norm_many_rows_equal_single_rows(fmt, K):
    """A row's result does not depend on the rows beside it or on its place."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(1203, K, generator=g, device=DEV).bfloat16()
    r = torch.randn(1203, K, generator=g, device=DEV).bfloat16()
    w = torch.randn(K, generator=g, device=DEV).bfloat16()
    q, s, h, y = lb.lowbit_add_rmsnorm_q8(x, w, 1e-6, fmt, residual=r, want_y=True)
    at = [0, 1, 63, 255, 256, 600, 1201, 1202]
    for m in at:
        q1, s1, h1, y1 = lb.lowbit_add_rmsnorm_q8(x[m:m + 1].clone(), w, 1e-6, fmt,
                                                  residual=r[m:m + 1].clone(), want_y=True)
        assert torch.equal(q1[0].view(torch.uint8), q[m].view(torch.uint8)) and torch.equal(s1[0], s[m])
        assert torch.equal(h1[0], h[m]) and torch.equal(y1[0], y[m])
    check_norm(x[at].cpu(), r[at].cpu(), w.cpu(), float(np.float32(1e-6)), fmt, q[at], s[at], h[at], y[at],
               "bf16")


@pytest.mark.parametrize("fmt", [lb.Q8_I8, lb.Q8_F8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [160, 2528, 4128, 33024])
def test_norm_extreme_rows(dtype, fmt, K):
    """Rows of zeros, a NaN, infinities, squares beyond fp32, tiny values; gains beyond the range."""
    rng = np.random.default_rng(K)
    x = torch.from_numpy(rng.standard_normal((10, K)).astype(np.float32))
    big = 3e4 if dtype == "f16" else 2e38
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, K - 1] = float("inf")
    x[3, :2] = torch.tensor([-float("inf"), float("inf")])
    x[4] *= big / 8
    x[5] = big
    x[6] = 0.0
    x[6, 77] = big
    x[7] *= 1e-7
    x[8] *= 0.0 if dtype == "f16" else 1e-30
    x = x.to(DT[dtype])
    for r in (None, torch.zeros_like(x)):
        q, s, h, y = lb.lowbit_add_rmsnorm_q8(x.to(DEV), None, 1e-5, fmt, want_y=True,
                                              residual=None if r is None else r.to(DEV))
        check_norm(x, r, None, float(np.float32(1e-5)), fmt, q, s, h, y, dtype)
    # x + residual overflows fp16: the stored infinity marks the row
    if dtype == "f16":
        a = torch.full((2, K), 100.0, dtype=torch.float16)
        a[0, 3] = 6e4
        b = a.clone()
        q, s, h, y = lb.lowbit_add_rmsnorm_q8(a.to(DEV), None, 1e-5, fmt, residual=b.to(DEV))
        check_norm(a, b, None, float(np.float32(1e-5)), fmt, q, s, h, y, dtype)
        assert torch.isnan(s[0]).all() and not torch.isnan(s[1]).any()


def test_norm_gain_not_finite_marks_its_span_only():
    K = 512
    x = torch.randn(3, K, device=DEV)
    g = torch.ones(K, device=DEV)
    g[200] = float("inf")
    q, s, _, _ = lb.lowbit_add_rmsnorm_q8(x, g, 1e-5, lb.Q8_F8)
    assert torch.equal(torch.isnan(s).cpu(), torch.tensor([[False, True, False, False]] * 3))
    assert (q.view(torch.uint8)[:, 128:256] == 0).all()
    q, s, _, _ = lb.lowbit_add_rmsnorm_q8(x, g, 1e-5, lb.Q8_I8)
    assert torch.isnan(s).all() and (q == 0).all()


@pytest.mark.parametrize("K", [160, 4096, 33024])
def test_norm_in_place_and_given_outputs(K):
    """The residual stream updated in place; outputs given by the caller are the ones returned."""
    x = torch.randn(37, K, device=DEV).bfloat16()
    r = torch.randn(37, K, device=DEV).bfloat16()
    w = torch.randn(K, device=DEV).bfloat16()
    want = lb.lowbit_add_rmsnorm_q8(x, w, 1e-5, lb.Q8_F8, residual=r, want_y=True)
    for inplace in ("residual", "x"):
        xi, ri = x.clone(), r.clone()
        h = ri if inplace == "residual" else xi
        out = [torch.empty_like(t) for t in (want[0], want[1], want[3])]
        got = lb.lowbit_add_rmsnorm_q8(xi, w, 1e-5, lb.Q8_F8, residual=ri, h=h, q=out[0], qscale=out[1], y=out[2])
        assert got[0] is out[0] and got[1] is out[1] and got[2] is h and got[3] is out[2]
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(xi if inplace == "residual" else ri, x if inplace == "residual" else r)


def test_norm_no_rows():
    x = torch.empty(0, 256, device=DEV, dtype=torch.float16)
    q, s, h, y = lb.lowbit_add_rmsnorm_q8(x, None, 1e-5, lb.Q8_F8, residual=x.clone(), want_y=True)
    assert q.shape == (0, 256) and s.shape == (0, 2) and h.shape == y.shape == (0, 256)


# ----------------------------------------------------------------- linear --

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 400, 1024, 1552])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 33, 64, 70])
def test_linear_small(dtype, K, M):
    for N, bias in [(1, False), (63, True), (130, False), (264, True)]:
        run_linear(M + K, M, N, K, dtype, bias)


@pytest.mark.parametrize("M, N, K, dtype, bias", [
    (1, 4096, 4096, "bf16", False), (3, 1000, 4112, "f16", True), (8, 4097, 8208, "f32", False),
    (16, 14336, 1024, "bf16", True), (20, 513, 14336, "f32", False), (48, 2050, 2064, "f16", False),
    (97, 1030, 1040, "f32", True), (128, 4096, 1024, "bf16", False), (129, 259, 4096, "f32", False),
    (200, 3000, 400, "f16", True), (257, 515, 784, "f32", False), (300, 4100, 272, "f32", True),
    (513, 1025, 1168, "bf16", True), (1025, 4099, 144, "f32", False), (2100, 2056, 272, "f16", False),
])
def test_linear_shapes(M, N, K, dtype, bias):
    run_linear(M + N + K, M, N, K, dtype, bias)


def exact_inputs(seed, M, N, K, E=None):
    """Small integers and powers of two: every sum is exact in fp32, in any order."""
    rng = np.random.default_rng(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    lead = () if E is None else (E,)
    ints = np.array([0x00, 0x38, 0x40, 0xb8, 0xc0, 0x30], np.uint8)     # 0, 1, 2, -1, -2, 0.5
    xq, wq = rng.choice(ints, (M, K)), rng.choice(ints, (*lead, N, K))
    xs = (2.0 ** rng.integers(-2, 2, (M, kb))).astype(np.float32)
    ws = (2.0 ** rng.integers(-2, 2, (*lead, nb, kb))).astype(np.float32)
    return xq, xs, wq, ws


@pytest.mark.parametrize("M, N, K", [(1, 300, 2064), (9, 4100, 400), (31, 257, 1040), (64, 640, 2048),
                                     (130, 390, 1168), (259, 771, 656), (700, 2310, 912), (1030, 4200, 272)])
def test_linear_exact(M, N, K):
    xq, xs, wq, ws = exact_inputs(M, M, N, K)
    ref, A = o.linear_f8(xq, xs, wq, ws)
    assert A.max() < 2 ** 18                   # steps of 2^-6: below 2^24 of them
    y = lb.lowbit_linear_f8(up8(xq), up(xs), up8(wq), up(ws), None, torch.float32)
    assert np.array_equal(f64(y), ref)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("M, N, K", [
    (12, 300, 8336), (20, 300, 4096), (31, 2000, 8208), (70, 300, 8208),     # K splits
    (512, 2050, 14336), (300, 4608, 3600),                # 128 x 128 tiles, in splits and whole
    (300, 28700, 272), (257, 28673, 16), (300, 28700, 400), (259, 28700, 8336), (512, 14336, 528),  # 256 x 256
    (1100, 14340, 1168), (300, 28700, 528), (600, 14340, 1040), (600, 14340, 1168), (4100, 16400, 144), (700, 28700, 656),
    (8192, 8192, 16), (300, 8200, 8208),
    (4, 11000, 16), (8, 12000, 144), (15, 14001, 272), (9, 13000, 1168),      # two groups of waves, odd K blocks
    (33, 4100, 1552), (130, 4000, 1296), (250, 4000, 1552), (128, 1030, 2064), (250, 4000, 2064),
    (600, 4000, 4112), (700, 4000, 3088),
])
def test_linear_variants(M, N, K, dtype):
    """Every kernel variant at ragged edges: exact inputs, every column near a tile's edge and a
    sample of the rest; twice with the same result; a workspace that is too small changes nothing."""
    xq, xs, wq, ws = exact_inputs(M + K, M, N, K)
    rng = np.random.default_rng(N)
    cols = np.unique(np.concatenate([np.arange(min(N, 20)), np.arange(max(0, N - 300), N),
                                     rng.integers(0, N, 200)]))
    bias = (rng.integers(-8, 9, N) * 0.5).astype(np.float32)
    ref, A = o.linear_f8(xq, xs, wq, ws, bias, cols)
    a = [up8(xq), up(xs), up8(wq), up(ws), up(bias).to(DT[dtype])]
    y = lb.lowbit_linear_f8(*a, DT[dtype])
    assert torch.equal(y, lb.lowbit_linear_f8(*a, DT[dtype]))
    assert A.max() < 2 ** 18                   # steps of 2^-6: below 2^24 of them, exact in fp32
    got = f64(y[:, torch.from_numpy(cols).to(DEV)])
    want = ref if dtype == "f32" else f64(torch.from_numpy(ref).to(DT[dtype]))
    assert np.array_equal(got, want)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    assert torch.equal(y, lb.lowbit_linear_f8(*a, DT[dtype], workspace=small))


def test_linear_split_on_another_stream():
    """The workspace made for a call lives on the call's stream."""
    xq, xs, wq, ws = exact_inputs(5, 64, 4096, 8192)
    a = [up8(xq), up(xs), up8(wq), up(ws)]
    want = lb.lowbit_linear_f8(*a, None, torch.float32)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    ys = [torch.zeros_like(want) for _ in range(12)]
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        s = streams[i % 3]
        lb.lowbit_linear_f8(*a, None, torch.float32, y=y, stream=s if i % 2 else s.cuda_stream)
        torch.empty(1 << 20, device=DEV).fill_(float("nan"))     # what a freed workspace might become
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("K", [144, 1040])
def test_linear_one_hot_reads_the_right_column(M, K):
    """Row m picks column (7 m) % K of the weight: y[m, n] = wq[n, k] exactly."""
    rng = np.random.default_rng(K)
    N = 300
    wq = random_codes(rng, (N, K))
    xq = np.zeros((M, K), np.uint8)
    cols = np.array([0, 15, 16, 127, 128, K - 1, K - 16, K - 17] + [(7 * m) % K for m in range(M)])[:M]
    xq[np.arange(M), cols] = 0x38
    y = lb.lowbit_linear_f8(up8(xq), torch.ones(M, -(-K // 128), device=DEV), up8(wq),
                            torch.ones(3, -(-K // 128), device=DEV), None, torch.float32)
    assert np.array_equal(f64(y), o.E4M3[wq[:, cols].T])


@pytest.mark.parametrize("M", [1, 20, 90, 300])
def test_linear_nan_stays_in_its_rows_and_columns(M):
    N, K = 200, 400
    xq, xs, wq, ws, _ = linear_inputs(M, M, N, K, "f32", False)
    ref, A = o.linear_f8(xq, xs, wq, ws)
    xq[M - 1, K - 1] = 0x7f                    # a NaN code in the last, partial block
    wq[130, 3] = 0xff
    xs[0, 1] = np.nan
    y = lb.lowbit_linear_f8(up8(xq), up(xs), up8(wq), up(ws), None, torch.float32)
    ref[[0, M - 1]] = np.nan
    ref[:, 130] = np.nan
    close(y, ref, A, 4, torch.float32, f"NaN M={M}")


def test_linear_nan_in_256_tiles():
    """The same through 256 x 256 tiles: codes and scales of NaN beside each edge of K's partial block."""
    M, N, K = 600, 14340, 1040
    xq, xs, wq, ws = exact_inputs(6, M, N, K)
    xq[599, K - 1], xq[255, K - 16], xq[300, 0] = 0x7f, 0xff, 0x7f
    wq[N - 1, K - 1], wq[255, K - 16], wq[256, 1023] = 0x7f, 0xff, 0x7f
    xs[31, 8], xs[512, 0], ws[5, 8] = np.nan, np.nan, np.nan
    cols = np.unique(np.concatenate([np.arange(250, 260), np.arange(630, 780), np.arange(N - 9, N)]))
    y = lb.lowbit_linear_f8(up8(xq), up(xs), up8(wq), up(ws), None, torch.float16)
    ref, _ = o.linear_f8(np.where(xq & 0x7f == 0x7f, 0, xq), np.nan_to_num(xs),
                         np.where(wq & 0x7f == 0x7f, 0, wq), np.nan_to_num(ws), None, cols)
    ref[[31, 255, 300, 512, 599]] = np.nan
    ref[:, (cols == N - 1) | (cols == 255) | (cols == 256) | (cols // 128 == 5)] = np.nan
    got = f64(y[:, torch.from_numpy(cols).to(DEV)])
    assert np.array_equal(got, f64(torch.from_numpy(ref).to(torch.float16)), equal_nan=True)
    assert int(torch.isnan(y).any(0).sum()) == N and int(torch.isnan(y).all(0).sum()) == 3 + 128
    assert int(torch.isnan(y).all(1).sum()) == 5


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_linear_unaligned_output_and_neighbours(dtype):
    """y at an odd element offset, N odd: nothing outside y is written."""
    M, N, K = 70, 131, 272
    xq, xs, wq, ws, b = linear_inputs(1, M, N, K, dtype, True)
    flat = torch.full((M * N + 64,), 5.0, dtype=DT[dtype], device=DEV)
    for off in (1, 3, 8):
        flat.fill_(5.0)
        y = flat[off:off + M * N].view(M, N)
        lb.lowbit_linear_f8(up8(xq), up(xs), up8(wq), up(ws), b.to(DEV), DT[dtype], y=y)
        ref, A = o.linear_f8(xq, xs, wq, ws, f64(b))
        close(y, ref, A, 3, DT[dtype], f"offset {off}")
        assert (flat[:off] == 5.0).all() and (flat[off + M * N:] == 5.0).all()


@pytest.mark.parametrize("M, N, K", [(1, 4096, 4096), (128, 1024, 4096), (300, 1000, 2064)])
def test_linear_is_deterministic_and_rows_agree(M, N, K):
    xq, xs, wq, ws, _ = linear_inputs(3, M, N, K, "bf16", False)
    a = [up8(xq), up(xs), up8(wq), up(ws)]
    y = [lb.lowbit_linear_f8(*a, None, torch.bfloat16) for _ in range(3)]
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_linear_no_rows():
    y = lb.lowbit_linear_f8(torch.empty(0, 256, device=DEV, dtype=F8), torch.empty(0, 2, device=DEV),
                            torch.zeros(40, 256, device=DEV).to(F8), torch.ones(1, 2, device=DEV), None,
                            torch.float16)
    assert y.shape == (0, 40)


def test_linear_weight_past_4_gib():
    """Byte offsets beyond 32 bits in the weights and beyond 2^31 elements of y's row index space."""
    N, K, M = 1 << 16, (1 << 16) + 128, 3
    wq = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    at = torch.tensor([0, 1, 40000, N - 1], device=DEV)
    wq[at] = (torch.arange(K, device=DEV) % 7 + 0x30).to(torch.uint8)
    ws = torch.ones(N // 128, K // 128, device=DEV)
    xq = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
    xq[:, K - 130:] = 0x38
    xq[1, 5] = 0x38
    for m in (M, 1):
        y = lb.lowbit_linear_f8(xq[:m].view(F8), torch.ones(m, K // 128, device=DEV), wq.view(F8), ws, None,
                                torch.float32)
        row = o.E4M3[(np.arange(K) % 7 + 0x30)]
        want = np.array([row[K - 130:].sum(), row[K - 130:].sum() + row[5], row[K - 130:].sum()])[:m]
        got = f64(y[:, at])
        assert np.allclose(got, want[:, None], rtol=0, atol=2 * 130 * U * np.abs(row).sum())
        y[:, at] = 0
        assert (y == 0).all()


@pytest.mark.parametrize("N, K, dtype, gather", [
    (256, 65664, "bf16", False), (256, 65664, "f32", False), (256, 65664, "bf16", True),   # xq past 4 GiB
    (40000, 1040, "f16", False), (40000, 144, "f16", False)])                              # y past 4 GiB
def test_linear_rows_past_4_gib(N, K, dtype, gather):
    """All rows zero but a few, whose exact products appear in their places alone."""
    M, kb = 66000, -(-K // 128)
    at = np.array([0, 1, 40000, 65535, 65536, 65600, M - 1])
    xs_, xsc, wq, ws = exact_inputs(N, len(at), N, K)
    if K > 8192:                               # sums below 2^24 steps of 2^-6 all the same
        xs_[:, 200:-200] = 0
    cols = np.unique(np.concatenate([np.arange(40), np.arange(N - 300, N)])) if N > 256 else None
    ref, A = o.linear_f8(xs_, xsc, wq, ws, None, *(() if cols is None else (cols,)))
    assert A.max() < 2 ** 18
    xq = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
    xs = torch.ones(M, kb, device=DEV)
    rows = torch.from_numpy(at).to(DEV)
    xq[rows] = torch.from_numpy(xs_).to(DEV)
    xs[rows] = up(xsc)
    if gather:
        y = lb.lowbit_linear_f8_grouped(xq.view(F8), xs, up(np.array([0, M], np.int32)), up8(wq[None]), up(ws[None]),
                                        None, DT[dtype], rows=torch.arange(M, dtype=torch.int32, device=DEV))
    else:
        y = lb.lowbit_linear_f8(xq.view(F8), xs, up8(wq), up(ws), None, DT[dtype])
    got = y[rows] if cols is None else y[rows][:, torch.from_numpy(cols).to(DEV)]
    assert np.array_equal(f64(got), f64(torch.from_numpy(ref).to(DT[dtype])))
    y[rows] = 0
    assert not y.any()


def test_norm_and_quantizer_past_4_gib():
    """Rows on both sides of 2^32 elements: a row's codes are those of the row alone."""
    M, K = 66000, 65664
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 32767, 65405, 65406, 65535, M - 1], device=DEV)
    x[at] = torch.randn(len(at), K, device=DEV).bfloat16()
    few = x[at]
    q, s = lb.lowbit_quantize_act_f8(x)
    q1, s1 = lb.lowbit_quantize_act_f8(few)
    assert torch.equal(q[at].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[at], s1)
    assert int((s != 0).any(1).sum()) == len(at)
    del q, s
    q, s, h, _ = lb.lowbit_add_rmsnorm_q8(x, None, 1e-5, lb.Q8_F8, residual=x)
    q1, s1, h1, _ = lb.lowbit_add_rmsnorm_q8(few, None, 1e-5, lb.Q8_F8, residual=few)
    assert torch.equal(q[at].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[at], s1)
    assert torch.equal(h[at], h1) and int((s != 0).any(1).sum()) == len(at)


# ---------------------------------------------------------------- grouped --

def run_grouped(seed, counts, M, N, K, dtype, gather=True, bias=False, first=0, behind=0, rows=None):
    """counts: rows of each expert; `first` rows before the first expert's, `behind` after the last."""
    rng = np.random.default_rng(seed)
    E = len(counts)
    off = (first + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    T = int(off[-1]) + behind
    if not gather:
        M = T
    xq, xs, wq, ws, b = linear_inputs(seed, M, N, K, dtype, bias, lead=(E,))
    if gather and rows is None:
        rows = rng.integers(0, M, T).astype(np.int32)
    y0 = torch.full((T, N), 3.0, dtype=DT[dtype])
    y = lb.lowbit_linear_f8_grouped(up8(xq), up(xs), up(off), up8(wq), up(ws), None if b is None else b.to(DEV),
                                    DT[dtype], rows=up(rows) if gather else None, y=y0.to(DEV))
    ref, A = o.linear_f8_grouped(xq, xs, rows if gather else None, off, wq, ws, None if b is None else f64(b),
                                 f64(y0))
    close(y, ref, A, xs.shape[1], DT[dtype], f"counts={counts[:8]} N={N} K={K} {dtype}")
    return y


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [3, 0, 0, 17, 16, 1], [64, 65, 0, 63], [0, 0, 0],
                                    [130, 2, 33, 0, 7, 129], [300, 0, 1]])
def test_grouped_counts(dtype, gather, counts):
    run_grouped(len(counts), counts, 11, 72, 272, dtype, gather, bias=True, first=2, behind=5)
    run_grouped(len(counts) + 1, counts, 11, 130, 128, dtype, gather)


@pytest.mark.parametrize("E", [63, 64, 65, 128, 200])
def test_grouped_many_experts(E):
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 4, E) * (rng.random(E) < 0.6)
    counts[-1] = 2
    run_grouped(E, counts.tolist(), 9, 40, 144, "f32", bias=True, behind=3)
    run_grouped(E, [0] * (E - 1) + [70], 9, 40, 144, "f16", gather=False)


@pytest.mark.parametrize("counts, N, K, dtype", [
    ([8] * 16, 1408, 2048, "bf16"), ([700, 3, 0, 290], 520, 656, "f32"), ([100, 156, 257, 31], 1030, 272, "f16"),
    ([1, 1, 1, 1, 1, 1, 1, 1], 2048, 4096, "bf16"), ([2000, 1, 0, 0], 264, 144, "f32")])
def test_grouped_shapes(counts, N, K, dtype):
    run_grouped(sum(counts), counts, 50, N, K, dtype)


@pytest.mark.parametrize("counts", [[5, 0, 9, 40], [200, 61, 0, 300]])
def test_grouped_exact_and_equal_to_dense(counts):
    N, K, M = 390, 1168, 33
    xq, xs, wq, ws = exact_inputs(1, M, N, K, E=4)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = np.random.default_rng(2).integers(0, M, off[-1]).astype(np.int32)
    y = lb.lowbit_linear_f8_grouped(up8(xq), up(xs), up(off), up8(wq), up(ws), None, torch.float32, rows=up(rows))
    for e in range(4):
        ref, _ = o.linear_f8(xq, xs, wq[e], ws[e])
        assert np.array_equal(f64(y[off[e]:off[e + 1]]), ref[rows[off[e]:off[e + 1]]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("counts, N, K", [
    ([30, 0, 25], 200, 4112), ([60, 0, 70], 300, 2064),   # K splits, 64 x 32 and 64 x 64
    ([100, 0, 61, 70], 2056, 2064), ([30, 9, 0, 52], 2056, 1552),             # two groups of waves
    ([400, 0, 500], 4000, 4112),
    ([200, 100, 0, 130], 6000, 272),                      # 128 x 128
    ([200, 100, 0, 290], 4100, 8208),                     # 128 x 128 in splits
    ([300, 260, 0, 208], 14356, 400), ([257, 1, 600, 0, 300], 14356, 144),
    ([2000, 988], 14356, 784), ([1, 730, 257], 14356, 528),                                 # 256 x 256
])
@pytest.mark.parametrize("gather", [True, False])
def test_grouped_variants(counts, N, K, dtype, gather):
    rng = np.random.default_rng(N + K)
    E, first, behind = len(counts), 3, 9
    off = (first + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    T = int(off[-1]) + behind
    M = 41 if gather else T
    xq, xs, wq, ws = exact_inputs(K, M, N, K, E=E)
    rows = rng.integers(0, M, T).astype(np.int32) if gather else None
    if gather:
        rows[[first, T - behind - 1]] = [-3, M]
    bias = (rng.integers(-8, 9, (E, N)) * 0.5).astype(np.float32)
    y0 = torch.full((T, N), 3.0, dtype=DT[dtype], device=DEV)
    a = [up8(xq), up(xs), up(off), up8(wq), up(ws), up(bias).to(DT[dtype]), DT[dtype]]
    r = up(rows) if gather else None
    y = lb.lowbit_linear_f8_grouped(*a, rows=r, y=y0.clone())
    cols = np.unique(np.concatenate([np.arange(min(N, 10)), np.arange(max(0, N - 280), N),
                                     rng.integers(0, N, 100)]))
    ref, A = o.linear_f8_grouped(xq, xs, rows, off, wq, ws, bias, f64(y0), cols)
    assert A.max() < 2 ** 18
    want = ref if dtype == "f32" else f64(torch.from_numpy(ref).to(DT[dtype]))
    assert np.array_equal(f64(y[:, torch.from_numpy(cols).to(DEV)]), want, equal_nan=True)
    assert (y[:first] == 3.0).all() and (y[T - behind:] == 3.0).all()
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    z = lb.lowbit_linear_f8_grouped(*a, rows=r, y=y0.clone(), workspace=small)
    assert torch.equal(y.nan_to_num(9.0), z.nan_to_num(9.0))


def test_grouped_rows_out_of_range_are_nan():
    counts, M = [4, 3, 70], 6
    rows = np.random.default_rng(0).integers(0, M, sum(counts)).astype(np.int32)
    rows[[0, 5, 30]] = [-1, M, np.iinfo(np.int32).max]
    rows[76] = np.iinfo(np.int32).min
    y = run_grouped(4, counts, M, 72, 272, "f32", rows=rows)
    assert torch.isnan(y[[0, 5, 30, 76]]).all()


@pytest.mark.parametrize("off", [[0, 50, 20, 90], [-7, 3, 200, 2 ** 31 - 1], [90, 0, 90, 0], [100, 100, 100, 100]])
def test_grouped_bad_offsets_stay_inside(off):
    """Offsets out of order or range: unspecified values inside y, nothing outside it."""
    T, N, K = 90, 72, 272
    xq, xs, wq, ws, _ = linear_inputs(0, T, N, K, "f32", False, lead=(3,))
    flat = torch.full((T * N + 4096,), 5.0, device=DEV)
    y = flat[2048:2048 + T * N].view(T, N)
    lb.lowbit_linear_f8_grouped(up8(xq), up(xs), up(np.array(off, np.int64).astype(np.int32)), up8(wq), up(ws),
                                None, torch.float32, y=y)
    assert (flat[:2048] == 5.0).all() and (flat[2048 + T * N:] == 5.0).all()


def test_grouped_same_index_twice_and_every_row_alike():
    rows = np.zeros(75, np.int32)
    y = run_grouped(9, [75], 4, 130, 400, "f32", rows=rows)
    assert torch.equal(y, y[:1].expand_as(y))


# ------------------------------------------- streams, graphs, the run together --

def moe_reference(x, gate_up, down, ids, w):
    """The block in float64 from the unquantized weights."""
    out = np.zeros_like(x)
    I = gate_up.shape[1] // 2
    for t in range(x.shape[0]):
        for e, r in zip(ids[t], w[t]):
            gu = gate_up[e] @ x[t]
            a = gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:]
            out[t] += r * (down[e] @ a)
    return out


@pytest.mark.parametrize("T", [1, 37])
def test_block_norm_router_experts(T):
    """Residual-add norm -> codes and y -> router on y -> experts on the codes, as a block runs."""
    torch.manual_seed(T)
    E, H, I, k = 6, 272, 144, 2
    gate_up, down = torch.randn(E, 2 * I, H) * 0.06, torch.randn(E, H, I) * 0.08
    m = lnn.F8Experts(E, H, I, dtype=torch.float32, device=DEV).set_weight(gate_up.to(DEV), down.to(DEV))
    x, r, g = torch.randn(T, H), torch.randn(T, H), 1 + 0.1 * torch.randn(H)
    router = torch.randn(E, H) * 0.1
    q, s, h, y = lb.lowbit_add_rmsnorm_q8(x.to(DEV), g.to(DEV), 1e-5, lb.Q8_F8, residual=r.to(DEV), want_y=True)
    w, ids = torch.softmax(y @ router.to(DEV).t(), -1).topk(k)
    out = m.forward_codes(q, s, ids, w)
    y64 = o.rmsnorm(f64(x + r), f64(g), 1e-5)
    assert np.abs(f64(y) - y64).max() <= 1e-5
    # the same products from the dequantized codes: only the intermediate codes' rounding is left
    deq = o.E4M3[patterns(q)] * np.repeat(f64(s), 128, 1)[:, :H]
    wd = [o.E4M3[patterns(c)] * np.repeat(np.repeat(f64(sc), 128, 1), 128, 2)[:, :c.shape[1], :c.shape[2]]
          for c, sc in ((m.gate_up, m.gate_up_scale), (m.down, m.down_scale))]
    ref = moe_reference(deq, wd[0], wd[1], ids.cpu().numpy(), f64(w))
    # an intermediate value is off by half an e4m3 step, 2^-4 of itself at most: |err| <= 2^-4 of
    # the sum of magnitudes of the down product, plus the fp32 terms (below a tenth of it)
    bound = np.zeros_like(ref)
    for t in range(T):
        for e, rw in zip(ids[t].tolist(), w[t].tolist()):
            gu = wd[0][e] @ deq[t]
            a = np.abs(gu[:I] / (1 + np.exp(-gu[:I])) * gu[I:])
            bound[t] += rw * (np.abs(wd[1][e]) @ np.maximum(a, a.max() * 2.0 ** -14))
    assert np.all(np.abs(f64(out) - ref) <= 1.1 * 2.0 ** -4 * bound)
    # the module's own forward quantizes y (fp32 here): the same codes, the same result
    assert torch.equal(m(y, ids, w), out)


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_experts_leave_padded_slots_out(kind):
    """Expert ids outside 0..E-1 add nothing, whatever memory their rows' buffers held before."""
    torch.manual_seed(8)
    E, H, I, T, k = 5, 144, 80, 33, 3
    m = lnn.F8Experts(E, H, I, device=DEV).set_weight(torch.randn(E, 2 * I, H, device=DEV) * 0.06,
                                                      torch.randn(E, H, I, device=DEV) * 0.08)
    x = torch.randn(T, H, device=DEV).bfloat16()
    ids, w = torch.randint(0, E, (T, k), device=DEV), torch.rand(T, k, device=DEV) + 0.1
    out = torch.rand(T, k, device=DEV) < 0.4
    out[0], out[1] = True, False
    padded = torch.where(out, torch.where(torch.rand(T, k, device=DEV) < 0.5, -1, E), ids).to(kind)
    want = m(x, ids, torch.where(out, 0.0, w))
    for n in (T * k * 2 * I, T * k * H):
        torch.full((n,), float("nan"), dtype=torch.bfloat16, device=DEV)
    got = m(x, padded, w)
    assert torch.equal(got, want) and (got[0] == 0).all() and (got[1] != 0).any()


@pytest.mark.parametrize("T", [1, 40, 700, 20000])
def test_experts_in_a_graph(T):
    """Replays with other tokens and routings, eager calls between them: each equal to the eager call."""
    torch.manual_seed(T)
    E, H, I, k = 16, 272, 144, 4
    m = lnn.F8Experts(E, H, I, device=DEV).set_weight(torch.randn(E, 2 * I, H, device=DEV) * 0.06,
                                                      torch.randn(E, H, I, device=DEV) * 0.08)

    def inputs():
        return (torch.randn(T, H, device=DEV).bfloat16(), torch.randint(-1, E, (T, k), device=DEV),
                torch.rand(T, k, device=DEV))

    x, ids, w = inputs()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        m(x, ids, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m(x, ids, w)
    for _ in range(6):
        new = inputs()
        for t, n in zip((x, ids, w), new):
            t.copy_(n)
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, m(*new))


def test_norm_feeds_both_linears():
    """int8 rows into lowbit_linear_a8, e4m3 blocks into lowbit_linear_f8."""
    torch.manual_seed(5)
    M, N, K = 24, 130, 416
    x, r, g = torch.randn(M, K).bfloat16(), torch.randn(M, K).bfloat16(), torch.randn(K).bfloat16()
    W = torch.randn(N, K) * 0.05
    a, asc, h, _ = lb.lowbit_add_rmsnorm_q8(x.to(DEV), g.to(DEV), 1e-5, lb.Q8_I8, residual=r.to(DEV))
    packed, s, z, codes = lb.lowbit_quantize_pack(W.to(DEV), 4, 32, torch.bfloat16, want_codes=True)
    y = lb.lowbit_linear_a8(a, asc, packed, s, z, None, 4, 32)
    ref, A = oracle.linear_a8(a.cpu().numpy(), asc.cpu().numpy(), codes.cpu().numpy(), s.float().cpu().numpy(),
                              z.float().cpu().numpy(), 32, None)
    assert np.all(np.abs(f64(y) - ref) <= oracle.tolerance(A))
    q, qs, h2, _ = lb.lowbit_add_rmsnorm_q8(x.to(DEV), g.to(DEV), 1e-5, lb.Q8_F8, residual=r.to(DEV))
    assert torch.equal(h, h2)
    wq, ws = lb.lowbit_quantize_weight_f8(W.to(DEV))
    y = lb.lowbit_linear_f8(q, qs, wq, ws, None, torch.bfloat16)
    ref, A = o.linear_f8(patterns(q), qs.cpu().numpy(), patterns(wq), ws.cpu().numpy())
    close(y, ref, A, 4, torch.bfloat16, "after the norm")


def block_calls(t):
    """Norm, dense linear, quantizer and grouped linear in a row on given outputs."""
    lb.lowbit_add_rmsnorm_q8(t["x"], t["g"], 1e-5, lb.Q8_F8, residual=t["r"], q=t["q"], qscale=t["qs"], h=t["h"])
    lb.lowbit_linear_f8(t["q"], t["qs"], t["wq"], t["ws"], None, torch.bfloat16, y=t["y"])
    lb.lowbit_quantize_act_f8(t["y"], t["yq"], t["ys"])
    lb.lowbit_linear_f8_grouped(t["yq"], t["ys"], t["off"], t["wg"], t["wgs"], None, torch.bfloat16,
                                rows=t["rows"], y=t["z"])


def block_tensors(seed, M):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, K, E, N2 = 1040, 2064, 5, 200
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    t = dict(x=rn(M, K).bfloat16(), r=rn(M, K).bfloat16(), g=rn(K).bfloat16())
    t["wq"], t["ws"] = lb.lowbit_quantize_weight_f8(rn(N, K) * 0.02)
    t["wg"], t["wgs"] = lb.lowbit_quantize_weight_f8(rn(E, N2, N) * 0.02)
    t["rows"] = torch.randint(0, M, (2 * M,), generator=g, device=DEV, dtype=torch.int32)
    t["off"] = torch.tensor([0, M // 2, M // 2, M, 2 * M - 1, 2 * M], dtype=torch.int32, device=DEV)
    em = lambda dt, *s: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
    t.update(q=em(F8, M, K), qs=em(torch.float32, M, 17), h=em(torch.bfloat16, M, K), y=em(torch.bfloat16, M, N),
             yq=em(F8, M, N), ys=em(torch.float32, M, 9), z=em(torch.bfloat16, 2 * M, N2))
    return t


OUTS = ("q", "qs", "h", "y", "yq", "ys", "z")


@pytest.mark.parametrize("M", [1, 24, 200])
def test_graph_replays_equal_eager(M):
    """Captured and replayed with new inputs, eager work and synchronizations in between."""
    t = block_tensors(M, M)
    block_calls(t)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block_calls(t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block_calls(t)
    for k in range(4):
        new = block_tensors(100 + k, M)
        for name in ("x", "r"):
            t[name].copy_(new[name])
        for name in OUTS:
            t[name].zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t[n].clone() for n in OUTS}
        block_calls(t)
        for n in OUTS:
            assert torch.equal(got[n].view(torch.uint8), t[n].view(torch.uint8)), (k, n)


def test_two_graphs_and_eager_calls_on_two_streams():
    """Two captured graphs of the same shapes, replayed at once on two streams."""
    sets = [block_tensors(s, 130) for s in (1, 2)]
    graphs = []
    for t in sets:
        block_calls(t)
        t["want"] = {n: t[n].clone() for n in OUTS}
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block_calls(t)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for t in sets:
            for n in OUTS:
                t[n].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for t in sets:
            for n in OUTS:
                assert torch.equal(t[n].view(torch.uint8), t["want"][n].view(torch.uint8)), n


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_of_a_call_on_a_stream_spare_the_current_stream(handle):
    """What the current stream freed while it still reads it is not given to a call on another."""
    s = torch.cuda.Stream()
    at = s.cuda_stream if handle else s
    x = torch.randn(2048, 4096, device=DEV).bfloat16()
    w = torch.randn(4096, 4096, device=DEV).bfloat16()
    xq, xs = lb.lowbit_quantize_act_f8(x)
    wq, ws = lb.lowbit_quantize_weight_f8(w)
    off = torch.tensor([0, 2048], dtype=torch.int32, device=DEV)
    calls = [lambda: lb.lowbit_linear_f8(xq, xs, wq, ws, None, torch.bfloat16, stream=at),
             lambda: lb.lowbit_linear_f8_grouped(xq, xs, off, wq[None], ws[None], None, torch.bfloat16, stream=at),
             lambda: lb.lowbit_add_rmsnorm_q8(x, None, 1e-5, lb.Q8_F8, residual=x, want_y=True, stream=at),
             lambda: lb.lowbit_quantize_act_f8(x, stream=at), lambda: lb.lowbit_quantize_weight_f8(w, stream=at)]
    big = torch.randn(8192, 8192, device=DEV)
    for call in calls:
        torch.cuda.synchronize()
        held = [torch.full((2048, 4096), 2.0, dtype=t, device=DEV) for t in (torch.bfloat16, torch.int8) * 2]
        slow = big @ big                      # the copies below wait for it
        copies = [t + 0 * slow[0, 0].nan_to_num(0.0).to(t.dtype) for t in held]
        del held
        out = call()
        torch.cuda.synchronize()
        assert all((c == 2).all() for c in copies)
        del out, copies


def test_explicit_stream_argument():
    t = block_tensors(3, 24)
    block_calls(t)
    want = t["y"].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = torch.zeros_like(want)
    lb.lowbit_linear_f8(t["q"], t["qs"], t["wq"], t["ws"], None, torch.bfloat16, y=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)


# ------------------------------------------------------------ torch layer --

def test_modules_and_ops_match_the_calls():
    torch.manual_seed(0)
    lin = torch.nn.Linear(272, 200).to(DEV)
    m = lnn.F8Linear.from_linear(lin)
    assert m.dtype == torch.float32
    x = torch.randn(2, 9, 272, device=DEV)
    y = m(x)
    xq, xs = lb.lowbit_quantize_act_f8(x.view(-1, 272))
    wq, ws = lb.lowbit_quantize_weight_f8(lin.weight.detach())
    want = lb.lowbit_linear_f8(xq, xs, wq, ws, lin.bias.detach(), torch.float32)
    assert y.shape == (2, 9, 200) and torch.equal(y.view(-1, 200), want)
    # strided inputs are laid out by the ops
    xt = torch.randn(272, 18, device=DEV).t()
    assert torch.equal(m(xt), m(xt.contiguous()))
    q, s, h = torch.ops.lowbit.add_rmsnorm_q8(x, x, None, 1e-5, lb.Q8_F8)
    q2, s2, h2, _ = lb.lowbit_add_rmsnorm_q8(x.view(-1, 272), None, 1e-5, lb.Q8_F8, residual=x.view(-1, 272))
    assert torch.equal(q.view(-1, 272).view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s.view(-1, 3), s2)
    assert torch.equal(h.view(-1, 272), h2)
    q, s = torch.ops.lowbit.rmsnorm_q8(x[..., :256], None, 1e-5, lb.Q8_I8)
    q2, s2, _, _ = lb.lowbit_add_rmsnorm_q8(x[..., :256].reshape(-1, 256).contiguous(), None, 1e-5, lb.Q8_I8)
    assert torch.equal(q.view(-1, 256), q2) and torch.equal(s.view(-1), s2)
    net = torch.nn.Sequential(torch.nn.Linear(272, 64), torch.nn.SiLU(), torch.nn.Linear(64, 32)).to(DEV)
    lnn.quantize_linears_f8(net)
    assert net(x).shape == (2, 9, 32)


def test_compiled_module_equals_eager():
    torch.manual_seed(1)
    m = lnn.F8Linear.from_linear(torch.nn.Linear(256, 96).to(DEV).bfloat16())
    x = torch.randn(5, 256, device=DEV).bfloat16()
    f = torch.compile(m, fullgraph=True, backend="aot_eager")
    assert torch.equal(f(x), m(x))


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 272, device=DEV, dtype=torch.bfloat16)
    with pytest.raises(lb.LowbitError, match="INVALID_ARG"):
        lb.lowbit_add_rmsnorm_q8(x, None, 0.0, lb.Q8_F8)
    with pytest.raises(lb.LowbitError, match="INVALID_ARG"):
        lb.lowbit_add_rmsnorm_q8(x, None, 1e-5, lb.Q8_I8)              # 272 is no multiple of 32
    with pytest.raises(ValueError, match="contiguous"):
        lb.lowbit_quantize_act_f8(torch.zeros(272, 4, device=DEV).t())
    with pytest.raises(ValueError, match="one device|GPU memory"):
        lb.lowbit_add_rmsnorm_q8(x, torch.zeros(272, dtype=torch.bfloat16), 1e-5, lb.Q8_F8)
