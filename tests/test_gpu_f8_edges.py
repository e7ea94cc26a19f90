"""The 8-bit path on the GPU at the ends of its ranges: huge rows, large grids, wide scales, the
accuracy of 16-bit outputs, and cast or shared modules."""
import numpy as np
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn
from oracle import f8_oracle as o

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24


def f64(t):
    return t.detach().double().cpu().numpy()


def patterns(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def up8(a):
    return up(a).view(F8)


# ------------------------------------------------------------------- norm --

@pytest.mark.parametrize("fmt", [lb.Q8_NONE, lb.Q8_I8, lb.Q8_F8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("waves", range(1, 18))
def test_norm_at_each_width(waves, dtype, fmt):
    """Every number of threads a row can take, at both ends of its widths and between: y within the
    oracle's bound (at most K / 64 + 32 additions in a row, halved by the root, and 8 roundings),
    whole rows and rows of a batch alike."""
    for K in (512 * (waves - 1) + 32, 512 * waves - 256, 512 * waves - 32):
        rng = np.random.default_rng(K)
        x = torch.from_numpy(rng.standard_normal((9, K)).astype(np.float32)).to(DT[dtype])
        g = torch.from_numpy(rng.standard_normal(K).astype(np.float32)).to(DT[dtype])
        q, s, h, y = lb.lowbit_add_rmsnorm_q8(x.to(DEV), g.to(DEV), 1e-5, fmt, want_y=True)
        ref = o.rmsnorm(f64(x), f64(g), float(np.float32(1e-5)))
        d = (K / 128 + 24) * U
        fi = torch.finfo(DT[dtype])
        half = np.maximum(np.abs(ref) * (1 + d) * fi.eps / 2, fi.smallest_normal * fi.eps / 2)
        assert np.all(np.abs(f64(y) - ref) <= d * np.abs(ref) + half)
        one = lb.lowbit_add_rmsnorm_q8(x[7:8].to(DEV), g.to(DEV), 1e-5, fmt, want_y=True)
        assert torch.equal(one[3][0], y[7])
        if fmt != lb.Q8_NONE:
            assert torch.equal(one[0][0].view(torch.uint8), q[7].view(torch.uint8)) and torch.equal(one[1][0], s[7])
            span = K if fmt == lb.Q8_I8 else 128
            codes = f64(q) if fmt == lb.Q8_I8 else o.E4M3[patterns(q)]
            top = 127.0 if fmt == lb.Q8_I8 else 448.0
            full = np.repeat(f64(s).reshape(9, -1), span, 1)[:, :K]
            step = 0.5 * full if fmt == lb.Q8_I8 else np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * full)
            assert np.all(np.abs(codes * full - ref) <= step * (1 + 2 * d) + 2 * d * np.abs(ref))
            assert all((np.abs(codes[:, b:b + span]).max(1) == top).all() for b in range(0, K, span))


def test_norm_codes_are_those_of_its_own_y():
    """With fp32 the unrounded y is the one returned: codes and scales are the oracle's rule on it,
    bit for bit."""
    for M, K in ((5, 160), (3, 1056), (2, 4128), (3, 8256), (2, 33024)):
        x, g = torch.randn(M, K, device=DEV) * 3, torch.randn(K, device=DEV)
        q, s, _, y = lb.lowbit_add_rmsnorm_q8(x, g, 1e-5, lb.Q8_F8, want_y=True)
        rq, rs = o.quantize_f8_rows(y.cpu().numpy())
        assert np.array_equal(patterns(q), rq) and np.array_equal(s.cpu().numpy(), rs)
        q, s, _, y = lb.lowbit_add_rmsnorm_q8(x, g, 1e-5, lb.Q8_I8, want_y=True)
        v = y.cpu().numpy()
        rs, f = o.span_scale(v, 127.0)
        assert np.array_equal(s.cpu().numpy(), rs)
        assert np.array_equal(q.cpu().numpy(), np.rint((v * f[:, None]).astype(np.float32)).astype(np.int8))


@pytest.mark.parametrize("K", [16, 1024, 2048, 4096, 16384, 32768, 65536])
def test_norm_rows_near_the_largest_number(K):
    """Rows of one value r above 2^126, whose reciprocal is subnormal: y = r / r.  r has five
    significant bits, so that every sum of its squares (K a power of two), their mean and its root
    are exact; what is left is the root's reciprocal and the product with it, each off by at most
    u, so y lies within 2 u of 1."""
    r = torch.tensor([k / 16.0 for k in range(17, 32)], dtype=torch.float64) * 2.0 ** 127
    x = r.float()[:, None].expand(-1, K).contiguous()
    x[1::2, ::2] *= -1.0
    for res in (None, torch.zeros_like(x)):
        q, s, h, y = lb.lowbit_add_rmsnorm_q8(x.to(DEV), None, 1e-5, lb.Q8_F8, want_y=True,
                                              residual=None if res is None else res.to(DEV))
        want = np.sign(x.numpy().astype(np.float64))
        assert np.abs(f64(y) - want).max() <= 2 * U
        assert np.abs(f64(s) * 448 - 1).max() <= 4 * U
        assert np.array_equal(o.E4M3[patterns(q)], 448 * want)


# -------------------------------------------------------------- quantizer --

def test_quantize_act_f8_of_the_most_blocks():
    """2^28 - 16 rows of one block each: the largest launch; every row as in a small call."""
    M, K, n = (1 << 28) - 16, 16, 1 << 12
    base = torch.randn(n, K, device=DEV).bfloat16()
    want, wants = lb.lowbit_quantize_act_f8(base)
    q, s = lb.lowbit_quantize_act_f8(base.repeat((1 << 28) // n, 1)[:M])
    whole = M // n * n
    q = q.view(torch.uint8)
    assert (q[:whole].view(-1, n, K) == want.view(torch.uint8)).all()
    assert (s[:whole].view(-1, n) == wants.view(-1)).all()
    assert torch.equal(q[whole:], want.view(torch.uint8)[:M - whole]) and torch.equal(s[whole:], wants[:M - whole])


# ----------------------------------------------------------------- linear --

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M, N, K", [(1, 11100, 8192), (16, 16300, 8192), (8, 12000, 8208), (3, 11000, 8064)])
def test_linear_few_rows_of_long_k(M, N, K, dtype):
    """Both sides of the rule for rows that lie a multiple of 8 KiB apart."""
    xq, xs, wq, ws = exact_inputs(M + K, M, N, K)
    cols = np.unique(np.concatenate([np.arange(70), np.arange(N - 300, N), np.random.default_rng(N).integers(0, N, 200)]))
    ref, A = o.linear_f8(xq, xs, wq, ws, None, cols)
    assert A.max() < 2 ** 18                   # steps of 2^-6: below 2^24 of them, exact in fp32
    y = lb.lowbit_linear_f8(up8(xq), up(xs), up8(wq), up(ws), None, DT[dtype])
    want = ref if dtype == "f32" else f64(torch.from_numpy(ref).to(DT[dtype]))
    assert np.array_equal(f64(y[:, torch.from_numpy(cols).to(DEV)]), want)


def grids_of_codes(rows, cols):
    """e4m3 codes 0 or 1 and a scale of 1, 2 or 4 a span, made in place (the arrays are large)."""
    q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV).random_(0, 2).mul_(0x38)
    return q.view(F8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_one_row_into_more_than_2_to_the_29_columns(dtype):
    """More blocks than 2^31 threads make; sums of at most 16 codes times scales up to 4, exact."""
    N, K = (1 << 29) + (1 << 20) + 37, 16
    wq, ws = grids_of_codes(N, K), (2.0 ** (torch.arange(-(-N // 128), device=DEV) % 3)).float()[:, None]
    xq = torch.tensor([[0x38, 0] * 8], dtype=torch.uint8, device=DEV).view(F8)
    y = lb.lowbit_linear_f8(xq, torch.ones(1, 1, device=DEV), wq, ws, None, DT[dtype])[0]
    for at in range(0, N, 1 << 24):
        n = min(1 << 24, N - at)
        want = wq[at:at + n].float()[:, ::2].sum(1) * ws[at // 128:, 0].repeat_interleave(128)[:n]
        assert torch.equal(y[at:at + n].float(), want), at


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_2_to_the_29_rows(dtype):
    """The other way round: rows past 2^29 into 16 columns."""
    M, K, N = (1 << 29) + 300, 16, 16
    xq, xs = grids_of_codes(M, K), (2.0 ** (torch.arange(M, dtype=torch.int32, device=DEV) % 3)).float()[:, None]
    wq = grids_of_codes(N, K)
    y = lb.lowbit_linear_f8(xq, xs, wq, torch.ones(1, 1, device=DEV), None, DT[dtype])
    w = wq.float().t().contiguous()
    for at in range(0, M, 1 << 24):
        n = min(1 << 24, M - at)
        assert torch.equal(y[at:at + n].float(), (xq[at:at + n].float() @ w) * xs[at:at + n]), at


def test_grouped_gather_past_4_gib_in_splits():
    """Rows gathered from more than 4 GiB of codes run in K splits through the workspace that the
    query asks for; without one the same sums (exact ones) come from one pass over K."""
    M, T, N, K = 226200, 3841, 2441, 19072
    rng = np.random.default_rng(4)
    few, xsc, wq, ws = exact_inputs(4, 48, N, K, E=2)
    few[rng.random((48, K)) < 0.9] = 0         # sums below 2^24 steps of 2^-6
    at = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 60)]))[:48]
    at[-1] = M - 1
    xq = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
    xs = torch.ones(M, K // 128, device=DEV)
    xq[up(at)], xs[up(at)] = up(few), up(xsc)
    pick = rng.integers(0, 48, T)
    off = np.array([0, 1700, T], np.int32)
    need = lb.lowbit_linear_f8_workspace_bytes(M, T, 2, N, K, torch.float16)
    assert need == 2 * T * 2444 * 4
    a = [xq.view(F8), xs, up(off), up8(wq), up(ws), None, torch.float16]
    rows = up(at[pick].astype(np.int32))
    y = lb.lowbit_linear_f8_grouped(*a, rows=rows)
    cols = np.unique(np.concatenate([np.arange(20), np.arange(N - 140, N), rng.integers(0, N, 60)]))
    for e in range(2):
        ref, A = o.linear_f8(few, xsc, wq[e], ws[e], None, cols)
        assert A.max() < 2 ** 18
        want = f64(torch.from_numpy(ref).to(torch.float16))[pick[off[e]:off[e + 1]]]
        assert np.array_equal(f64(y[off[e]:off[e + 1]][:, up(cols)]), want)
    small = torch.empty(256, dtype=torch.uint8, device=DEV)
    assert torch.equal(lb.lowbit_linear_f8_grouped(*a, rows=rows, workspace=small), y)


def cut_of_eights(x, w):
    """Mean square, per output, of what the fp8 instruction cuts off: each eight products lose at
    most seven parts below 2^-13 of their largest, of either sign, evenly spread at worst: a mean
    square of 7 / 3 (2^-13 max)^2, independent from one eight to the next."""
    top = (x[:, None, :] * w[None, :, :]).abs_().view(x.shape[0], w.shape[0], -1, 8).amax(3).double()
    return (7 / 3) * (2.0 ** -13 * top).square().sum(2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("M, N, K", [(3, 2000, 4096), (16, 8192, 2048), (64, 4096, 4096), (200, 2500, 2064),
                                     (600, 4000, 4112), (600, 14340, 1040)])
def test_16_bit_outputs_lose_no_more_than_the_cuts(M, N, K, dtype):
    """Every kernel family on random codes: the mean square error of the outputs is at most that of
    their rounding plus that of the instruction's cuts (a quarter more for the sample's spread).
    A lost product would break it from one output in 500 on (fp16) or in 50 (bf16, whose rounding's
    mean square, (1.66e-3 y)^2, is 1 / 88 of a product's y^2 / K at K = 4096)."""
    gen = torch.Generator(device=DEV).manual_seed(M + N)
    x = torch.randn(M, K, generator=gen, device=DEV)
    x[torch.rand(M, K, generator=gen, device=DEV) < 0.01] *= 20
    xq, xs = lb.lowbit_quantize_act_f8(x)
    wq, ws = lb.lowbit_quantize_weight_f8(torch.randn(N, K, generator=gen, device=DEV) * 0.02)
    y = lb.lowbit_linear_f8(xq, xs, wq, ws, None, DT[dtype])
    at = torch.unique(torch.randint(0, M, (24,), generator=gen, device=DEV))
    cols = torch.unique(torch.cat([torch.randint(0, N, (300,), generator=gen, device=DEV),
                                   torch.arange(N - 100, N, device=DEV)]))
    deq = xq[at].double() * xs[at].double().repeat_interleave(128, 1)[:, :K]
    wd = wq.view(torch.uint8)[cols].view(F8).double() * ws.double()[cols // 128].repeat_interleave(128, 1)[:, :K]
    ref = deq @ wd.t()
    rounding = (ref.to(DT[dtype]).double() - ref).square().mean()
    cuts = torch.cat([cut_of_eights(deq[i:i + 4].float(), wd.float()) for i in range(0, len(at), 4)]).mean()
    bound = 1.25 * (rounding + cuts)
    got = y[at][:, cols].double()
    assert (got - ref).square().mean() <= bound
    one = (deq.square() @ wd.square().t() / K).mean()                      # one product's mean square
    assert one / (500 if dtype == "f16" else 50) > bound


VARIANTS = [(3, 300, 400), (64, 640, 2048), (200, 2500, 1040), (600, 14340, 528), (600, 14340, 1040)]


@pytest.mark.parametrize("M, N, K", VARIANTS)
def test_scales_whose_product_is_at_the_ends_of_fp32(M, N, K):
    """Exact sums times 2^e, e the exponent of xscale * wscale: exact inside the normal range, off
    by less than 2^-125 a block below it, infinite or NaN past it."""
    xq, xs, wq, ws = exact_inputs(M, M, N, K)
    cols = np.unique(np.concatenate([np.arange(20), np.arange(N - 260, N)]))
    ref, A = o.linear_f8(xq, xs, wq, ws, None, cols)       # scale products of 2^-4 .. 2^2
    assert A.max() < 2 ** 18
    xq, wq, pick = up8(xq), up8(wq), up(cols)
    for dtype in (torch.float32, torch.bfloat16):
        # exponents of xscale and wscale: e = -117 keeps every product and sum normal, above 0 all finite
        for ex, ew in ((-100, -17), (-17, -100), (70, 37), (107, 0), (-120, 115)):
            y = lb.lowbit_linear_f8(xq, up(xs * np.float32(2.0 ** ex)), wq, up(ws * np.float32(2.0 ** ew)), None, dtype)
            want = torch.from_numpy(ref * 2.0 ** (ex + ew)).to(dtype)
            assert np.array_equal(f64(y[:, pick]), f64(want)), (ex, ew)
        for ex, ew in ((-70, -70), (-90, -50), (-119, -119)):
            y = lb.lowbit_linear_f8(xq, up(xs * np.float32(2.0 ** ex)), wq, up(ws * np.float32(2.0 ** ew)), None, dtype)
            err = np.abs(f64(y[:, pick]) - ref * 2.0 ** (ex + ew))
            half = np.maximum(np.abs(ref) * 2.0 ** (ex + ew) * torch.finfo(dtype).eps / 2, 2.0 ** -134)
            assert np.all(err <= xs.shape[1] * 2.0 ** -125 + half), (ex, ew)
        y = lb.lowbit_linear_f8(xq, up(xs * np.float32(2.0 ** 70)), wq, up(ws * np.float32(2.0 ** 70)), None, dtype)
        assert not torch.isfinite(y).any()


@pytest.mark.parametrize("M, dtype", [(1, "f32"), (3, "f16"), (16, "bf16"), (40, "f32"), (300, "f32"), (300, "f16"),
                                     (600, "bf16")])
def test_linear_of_a_weight_past_4_gib(M, dtype):
    """Weight rows on both sides of 2^32 bytes through few-row, tile and 256 x 256 kernels: exact
    sums of random codes all along K where rows are marked, zeros everywhere else."""
    N, K = 1 << 16, (1 << 16) + 128
    rng = np.random.default_rng(M)
    at = np.unique(np.concatenate([[0, 1, 127, 128, 32640, 65407, 65408, N - 1], rng.integers(0, N, 40)]))
    xq, xs, few, _ = exact_inputs(M, M, len(at), K)
    ws = (2.0 ** rng.integers(-2, 2, (N // 128, K // 128))).astype(np.float32)
    few[rng.random(few.shape) < 0.97] = 0      # sums below 2^24 steps of 2^-6
    wq = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    wq[up(at)] = up(few)
    y = lb.lowbit_linear_f8(up8(xq), up(xs), wq.view(F8), up(ws), None, DT[dtype])
    x, w, ref, A = o.E4M3[xq], o.E4M3[few], 0.0, 0.0
    for b in range(K // 128):                  # (each marked row with its own block's scales)
        k, s = np.s_[:, 128 * b:128 * b + 128], xs[:, b:b + 1] * ws[at // 128, b]
        ref, A = ref + s * (x[k] @ w[k].T), A + s * (np.abs(x[k]) @ np.abs(w[k]).T)
    assert A.max() < 2 ** 18
    want = f64(torch.from_numpy(ref).to(DT[dtype]))
    assert np.array_equal(f64(y[:, up(at)]), want)
    y[:, up(at)] = 0
    assert not y.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M, N, K", [(13, 4096, 4096), (100, 1024, 4096), (128, 4096, 14336), (300, 1000, 2064),
                                     (700, 4000, 1040), (600, 14340, 1040)])
def test_linear_equal_rows_give_equal_rows(M, N, K, dtype):
    """The same row everywhere: every row of y has the same bits, whatever tile it lies in."""
    gen = torch.Generator(device=DEV).manual_seed(K)
    xq, xs = lb.lowbit_quantize_act_f8(torch.randn(1, K, generator=gen, device=DEV))
    wq, ws = lb.lowbit_quantize_weight_f8(torch.randn(N, K, generator=gen, device=DEV))
    xq = xq.view(torch.uint8).expand(M, -1).contiguous().view(F8)
    y = lb.lowbit_linear_f8(xq, xs.expand(M, -1).contiguous(), wq, ws, None, DT[dtype])
    assert torch.equal(y, y[:1].expand_as(y)) and torch.isfinite(y).all() and (y != 0).any()


# ---------------------------------------------------------------- modules --

def test_cast_modules_compute_in_the_new_type():
    """A cast module equals the one made in that type: the same codes, scales and bias."""
    torch.manual_seed(3)
    lin = torch.nn.Linear(272, 200).to(DEV)
    lin.bias.data = lin.bias.data.bfloat16().float()
    x = torch.randn(7, 272, device=DEV).half()
    m = lnn.F8Linear.from_linear(lin, torch.bfloat16)
    want = lnn.F8Linear.from_linear(lin, torch.float16)(x)
    got = m.half()(x)
    assert got.dtype == torch.float16 and torch.equal(got, want)
    e = lnn.F8Experts(3, 144, 80, device=DEV).set_weight(torch.randn(3, 160, 144, device=DEV) * 0.06,
                                                         torch.randn(3, 144, 80, device=DEV) * 0.08)
    x = torch.randn(9, 144, device=DEV).half()
    ids, w = torch.randint(0, 3, (9, 2), device=DEV), torch.rand(9, 2, device=DEV)
    f = lnn.F8Experts(3, 144, 80, dtype=torch.float16, device=DEV)
    f.load_state_dict(e.state_dict())
    y = e.cpu().half().to(DEV)(x, ids, w)
    assert y.dtype == torch.float16 and torch.equal(y, f(x, ids, w))
