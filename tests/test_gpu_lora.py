"""Low-rank adapters on the GPU against the 64-bit oracle.

Tolerance, from the arithmetic (u = 2^-24, half a step of fp32; a sum in fp32 of terms a_i in a chain
of n additions is off by at most 2 n u sum |a_i|, where the matrix core truncates, too):
  * t = x A^T: a wave adds K / 32 steps of 32 products or fewer, then the waves and the K ranges meet
    (at most 16 + 64 additions): n1 = K / 32 + 32 + 80, one more rounding for the scale;
  * t as hi + lo: 2^-16 of it in bf16 (two halves of 8 bits each), 2^-22 in fp16 and 2^-25 of the
    row's largest |t| where lo falls among fp16's subnormal numbers;
  * t B^T: 2 (rank / 32 + 1) steps of 32, n2 = 2 rank / 32 + 34; the base's addition and the power of
    two's product: 2 u (|y| + |delta|);
  * half a step of y's type.
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
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _lib(lowbit_lib):
    return lowbit_lib


def f64(t):
    return t.detach().double().cpu().numpy()


def tolerance(ref, At, Ab, Am, K, rank, dtype):
    n1, n2 = K / 32 + 112, 2 * rank / 32 + 34
    pair = {torch.float32: 0.0, torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -16}[dtype]
    tol = (2 * n1 + 1) * U * At + (pair + 2 * n2 * U) * Ab + 4 * U * (np.abs(ref) + Ab)
    if dtype == torch.float16:
        tol += 2.0 ** -25 * Am
    fi = torch.finfo(dtype)
    return 1.001 * (tol + np.maximum(np.abs(ref) + tol, float(fi.tiny)) * (fi.eps / 2))


def inputs(seed, M, L, rank, K, N, dtype, ids=None, bare=0.2):
    g = torch.Generator().manual_seed(seed)

    def n(*shape):
        return torch.randn(*shape, generator=g)

    dt = DT[dtype]
    if ids is None:
        ids = torch.randint(0, L, (M,), generator=g)
        ids = torch.where(torch.rand(M, generator=g) < bare, torch.randint(0, 2, (M,), generator=g) * (L + 1) - 1, ids)
    return dict(x=n(M, K).to(dt), a=(n(L, rank, K) / K ** 0.5).to(dt), b=(n(L, N, rank) * 0.2).to(dt),
                scales=torch.rand(L, generator=g) + 0.5, base=n(M, N).to(dt), ids=ids.to(torch.int32), L=L)


def plan(t):
    rows, offsets, _ = lb.lowbit_group_rows(t["ids"].to(DEV).view(-1, 1), t["L"])
    return rows, offsets


def call(t, base=True, scales=True, rows=None, offsets=None, **kw):
    if offsets is None:
        rows, offsets = plan(t)
    return lb.lowbit_lora(t["x"].to(DEV), t["a"].to(DEV), t["b"].to(DEV), t["scales"].to(DEV) if scales else None,
                          rows, offsets, t["base"].to(DEV) if base else None, **kw)


def check(t, y, base=True, scales=True):
    ref, At, Ab, Am = o.lora(f64(t["x"]), f64(t["a"]), f64(t["b"]), f64(t["scales"]) if scales else None,
                             t["ids"].numpy(), f64(t["base"]) if base else None)
    tol = tolerance(ref, At, Ab, Am, t["x"].shape[1], t["a"].shape[1], t["x"].dtype)
    err = np.abs(f64(y) - ref)
    assert np.all(err <= tol), f"worst {np.max(err / tol)} at {np.argwhere(err > tol)[:5].tolist()}"
    off = (t["ids"].numpy() < 0) | (t["ids"].numpy() >= t["L"])
    if base:
        assert torch.equal(y.cpu()[torch.from_numpy(off)], t["base"][torch.from_numpy(off)])
    else:
        assert (y.cpu()[torch.from_numpy(off)] == 0).all()


SHAPES = [(1, 1, 8, 16, 1), (1, 4, 16, 4096, 4096), (2, 2, 16, 144, 33), (5, 3, 8, 48, 300), (16, 1, 32, 256, 256),
          (17, 5, 24, 272, 200), (33, 40, 16, 528, 129), (64, 32, 16, 1024, 520), (100, 1, 64, 400, 264),
          (130, 2, 48, 2064, 97), (200, 3, 128, 304, 640), (77, 2, 256, 512, 272), (300, 2, 136, 96, 1000),
          (700, 4, 40, 112, 24), (513, 1, 8, 32, 8)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, L, rank, K, N", SHAPES)
def test_lora(M, L, rank, K, N, dtype):
    t = inputs(M + rank + N, M, L, rank, K, N, dtype)
    check(t, call(t))


SCHEDULES = [  # one launch: one and two turns of columns, ranks to 32
             (16, 1, 16, 272, 2600), (200, 40, 16, 2064, 2100), (300, 80, 8, 144, 5200), (9, 3, 32, 4112, 700),
             (90, 30, 24, 528, 3300), (60, 30, 32, 144, 9000),
             # two launches of 16 rows a tile: long K in ranges, ranks past a pass
             (40, 20, 64, 4112, 300), (20, 20, 128, 2064, 520), (50, 2, 256, 1040, 129), (17, 17, 96, 16400, 40),
             (33, 20, 16, 16400, 40),
             # more adapters than a wave looks through at a time
             (150, 300, 16, 272, 200), (400, 700, 64, 144, 264), (70, 63, 8, 48, 24), (90, 255, 8, 16, 40),
             # of 64 and of 128, every number of rank tiles, whole tiles and parts, many turns of columns
             (128, 1, 16, 528, 1300), (192, 2, 32, 144, 2600), (256, 4, 72, 1040, 520), (600, 2, 16, 1040, 264),
             (600, 2, 24, 272, 1032), (1024, 2, 64, 2064, 520), (700, 2, 256, 272, 272), (900, 3, 8, 16, 5),
             (515, 1, 200, 4112, 65)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M, L, rank, K, N", SCHEDULES)
def test_lora_schedules(M, L, rank, K, N, dtype):
    t = inputs(M * 3 + rank + N, M, L, rank, K, N, dtype, bare=0.0 if M % 2 == 0 else 0.1)
    y = call(t)
    check(t, y)
    rows, offsets = plan(t)
    own = t["base"].to(DEV)                            # in place: the same
    lb.lowbit_lora(t["x"].to(DEV), t["a"].to(DEV), t["b"].to(DEV), t["scales"].to(DEV), rows, offsets, own, y=own)
    assert torch.equal(own, y)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_lora_without_base_or_scales(dtype):
    for M, L, rank, K, N in ((3, 2, 16, 64, 40), (150, 2, 64, 272, 250)):
        t = inputs(M, M, L, rank, K, N, dtype)
        check(t, call(t, base=False, scales=False), base=False, scales=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [96, 99])
def test_lora_in_place_and_off_alignment(dtype, N):
    t = inputs(8, 90, 3, 16, 272, N, dtype)
    want = call(t)
    rows, offsets = plan(t)
    y = t["base"].to(DEV)
    got = lb.lowbit_lora(t["x"].to(DEV), t["a"].to(DEV), t["b"].to(DEV), t["scales"].to(DEV), rows, offsets, y, y=y)
    assert got is y and torch.equal(y, want)
    flat = torch.full((92 * N + 1,), 5.0, dtype=DT[dtype], device=DEV)
    y = flat[1 + N:1 + 91 * N].view(90, N)
    call(t, y=y)
    assert torch.equal(y, want) and (flat[:1 + N] == 5).all() and (flat[1 + 91 * N:] == 5).all()


def test_lora_rows_as_they_stand():
    """No rows: positions are rows; heads and tails without an adapter, empty adapters."""
    M, L = 75, 5
    offsets = torch.tensor([4, 4, 37, 38, 38, 70], dtype=torch.int32)
    ids = torch.full((M,), -1)
    for l in range(L):
        ids[offsets[l]:offsets[l + 1]] = l
    t = inputs(5, M, L, 16, 160, 72, "bf16", ids=ids)
    y = call(t, offsets=offsets.to(DEV))
    check(t, y)
    own = t["base"].to(DEV)
    lb.lowbit_lora(t["x"].to(DEV), t["a"].to(DEV), t["b"].to(DEV), t["scales"].to(DEV), None, offsets.to(DEV), own,
                   y=own)
    assert torch.equal(own, y)


def test_lora_all_or_none_have_an_adapter():
    for v in (0, 2, -1):
        t = inputs(6, 40, 3, 16, 64, 48, "f16", ids=torch.full((40,), v))
        check(t, call(t))


def test_lora_rows_named_in_part_and_out_of_range():
    """Rows that are not named keep what y holds; indexes that are no row are left out."""
    t = inputs(7, 20, 2, 8, 32, 40, "bf16", ids=torch.tensor([0] * 10 + [1] * 10))
    rows = torch.tensor([3, 20, -1, 5, 12, 2 ** 31 - 1, 15, 1], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 4, 7], dtype=torch.int32, device=DEV)     # row 1: without an adapter
    y = torch.full((20, 40), 9.0, dtype=torch.bfloat16, device=DEV)
    call(t, rows=rows, offsets=offsets, y=y)
    want = call(t)
    named = [3, 5, 12, 15]
    assert torch.equal(y[named], want[named]) and torch.equal(y[1].cpu(), t["base"][1])
    rest = [i for i in range(20) if i not in named + [1]]
    assert (y[rest] == 9).all()


@pytest.mark.parametrize("offsets", [[-5, 100, 200], [3, 1, 2], [0, 2 ** 31 - 1, -2 ** 31], [9, 9, 9],
                                     [20, 0] * 100, [-2 ** 31, 2 ** 31 - 1, 7] * 100])
def test_lora_bad_offsets_stay_inside(offsets):
    """Unspecified values in y, its neighbours untouched."""
    t = inputs(7, 20, len(offsets) - 1, 8, 32, 40, "bf16")
    flat = torch.full((22 * 40,), 5.0, dtype=torch.bfloat16, device=DEV)
    call(t, rows=torch.arange(20, dtype=torch.int32, device=DEV),
         offsets=torch.tensor(offsets, dtype=torch.int32, device=DEV), y=flat[40:21 * 40].view(20, 40))
    torch.cuda.synchronize()
    assert (flat[:40] == 5).all() and (flat[21 * 40:] == 5).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M", [3, 100])
def test_lora_not_finite_stays_in_its_row(M, dtype):
    t = inputs(11, M, 1, 16, 64, 40, dtype, ids=torch.zeros(M, dtype=torch.int64))
    want = call(t)
    t["x"][1, 5] = NAN
    t["base"][2, 7] = INF
    y = call(t)
    assert torch.isnan(y[1]).all() and y[2, 7] == INF
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(y[keep], want[keep])
    cols = [i for i in range(40) if i != 7]
    assert torch.equal(y[2][cols], want[2][cols])


@pytest.mark.parametrize("power", [-40, 0, 40])
def test_lora_f16_intermediate_leaves_fp16(power):
    """x A^T far outside fp16, brought back by the scale: only y has to fit."""
    M, rank, K, N = 37, 16, 128, 48
    t = inputs(12, M, 1, rank, K, N, "f16", ids=torch.zeros(M, dtype=torch.int64))
    t["x"] = (t["x"].float() * 1000).half()
    t["a"] = (t["a"].float() * 1000).half()          # |t| near 1e6
    t["b"] = (t["b"].float() * 2.0 ** -14).half()
    t["scales"] = torch.tensor([2.0 ** (power - 8)])
    if power == 40:
        t["b"] = torch.zeros_like(t["b"])
        t["b"][:, :, 3] = 2.0 ** -24                 # the smallest number
    t["base"] = torch.zeros_like(t["base"]) if power < 0 else t["base"]
    y, At, Ab, Am = o.lora(f64(t["x"]), f64(t["a"]), f64(t["b"]), f64(t["scales"]), t["ids"].numpy(), f64(t["base"]))
    got = f64(call(t))
    tol = tolerance(y, At, Ab, Am, K, rank, torch.float16)
    fits = np.abs(y) < 65000
    assert np.all(np.abs(got - y)[fits] <= tol[fits]) and not np.isnan(got).any()


def test_lora_exact():
    """Small integers: every sum is exact, for every tile of rows, rank and type."""
    g = torch.Generator().manual_seed(2)
    for dtype in ("f32", "f16", "bf16"):
        for M, L, rank, K, N in ((1, 1, 16, 64, 64), (40, 3, 24, 96, 70), (600, 2, 64, 112, 300)):
            x = torch.randint(-1, 2, (M, K), generator=g) * (torch.rand(M, K, generator=g) < 0.1)
            a = torch.randint(-1, 2, (L, rank, K), generator=g) * (torch.rand(L, rank, K, generator=g) < 0.2)
            b = torch.randint(-1, 2, (L, N, rank), generator=g) * (torch.rand(L, N, rank, generator=g) < 0.3)
            base = torch.randint(-8, 9, (M, N), generator=g)
            ids = torch.randint(-1, L, (M,), generator=g)
            t = {k: v.to(DT[dtype]) for k, v in dict(x=x, a=a, b=b, base=base).items()}
            t.update(scales=torch.tensor([1.0, 2.0, 0.5])[:L], ids=ids.to(torch.int32), L=L)
            ref = o.lora(f64(t["x"]), f64(t["a"]), f64(t["b"]), f64(t["scales"]), ids.numpy(), f64(t["base"]))[0]
            assert np.abs(ref).max() <= 128
            assert np.array_equal(f64(call(t)), ref)


def test_lora_is_deterministic_and_rows_agree():
    t = inputs(3, 260, 4, 32, 528, 200, "bf16")
    y = call(t)
    for _ in range(3):
        assert torch.equal(call(t), y)
    # the same rows in another order within their adapters: the same values
    rows, offsets = plan(t)
    r, off = rows.cpu(), offsets.tolist()
    for lo, hi in zip(off[:-1], off[1:]):
        r[lo:hi] = r[lo:hi].flip(0)
    assert torch.equal(call(t, rows=r.to(DEV), offsets=offsets), y)


def test_lora_past_4_gib():
    """Rows of x and y, and adapters, whose offsets pass 32 bits."""
    K, N, M = 16384, 16, (1 << 32) // 16384 + 40
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    at = [0, M // 2 + 5, M - 1]
    for i, r in enumerate(at):
        x[r, i] = 1.0
        ids[r] = 0
    a = torch.zeros(1, 8, K, dtype=torch.bfloat16, device=DEV)
    a[0, 0, :3] = torch.tensor([2.0, 3.0, 5.0])
    b = torch.ones(1, N, 8, dtype=torch.bfloat16, device=DEV)
    rows, offsets, _ = lb.lowbit_group_rows(ids.view(-1, 1), 1)
    y = lb.lowbit_lora(x, a, b, None, rows, offsets, None)
    assert [y[r, 3].item() for r in at] == [2.0, 3.0, 5.0] and y.float().abs().sum().item() == 10.0 * N
    del x, y
    # y past 4 GiB: N large, few columns differ
    K, N, M = 16, 1 << 20, 4200
    x = torch.ones(M, K, dtype=torch.bfloat16, device=DEV)
    a, b = torch.ones(1, 8, K, dtype=torch.bfloat16, device=DEV), torch.ones(1, N, 8, dtype=torch.bfloat16, device=DEV)
    y = lb.lowbit_lora(x, a, b, None, None, torch.tensor([0, M], dtype=torch.int32, device=DEV), None)
    assert y.min().item() == 128.0 and y.max().item() == 128.0
    del x, y, b
    # adapters past 4 GiB
    L, rank, K, N = 1100, 128, 16384, 16
    a = torch.zeros(L, rank, K, dtype=torch.bfloat16, device=DEV)
    a[L - 1, 127, K - 1] = 4.0
    b = torch.ones(L, N, rank, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(3, K, dtype=torch.bfloat16, device=DEV)
    rows, offsets, _ = lb.lowbit_group_rows(torch.tensor([[5], [L - 1], [0]], device=DEV), L)
    y = lb.lowbit_lora(x, a, b, None, rows, offsets, None)
    assert (y[1] == 4).all() and (y[[0, 2]] == 0).all()


def test_lora_no_rows():
    t = inputs(3, 4, 2, 8, 32, 40, "bf16")
    x = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)
    y = lb.lowbit_lora(x, t["a"].to(DEV), t["b"].to(DEV), None, None, torch.zeros(3, dtype=torch.int32, device=DEV),
                       None)
    assert y.shape == (0, 40)


def test_lora_in_graphs_and_on_two_streams():
    """Two captured graphs and eager calls between their replays, each with its own workspace."""
    ts = [inputs(21, 70, 4, 32, 2064, 200, "bf16"), inputs(22, 300, 2, 64, 1040, 264, "bf16")]
    dev = [{k: v.to(DEV) for k, v in t.items() if torch.is_tensor(v)} for t in ts]
    outs, graphs = [], []

    def one(t, L):
        rows, offsets, _ = lb.lowbit_group_rows(t["ids"].view(-1, 1), L)
        return lb.lowbit_lora(t["x"], t["a"], t["b"], t["scales"], rows, offsets, t["base"])

    for t, d in zip(ts, dev):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            one(d, t["L"])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(one(d, t["L"]))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        news = [inputs(50 + 2 * i, 70, 4, 32, 2064, 200, "bf16"), inputs(51 + 2 * i, 300, 2, 64, 1040, 264, "bf16")]
        for d, n in zip(dev, news):
            for k in ("x", "ids", "base"):
                d[k].copy_(n[k])
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = [one(d, t["L"]) for d, t in zip(dev, ts)]
        torch.cuda.synchronize()
        for got, want in zip(outs, eager):
            assert torch.equal(got, want)


def test_lora_explicit_workspace_and_stream():
    t = inputs(30, 50, 3, 16, 1040, 96, "f16")
    want = call(t)
    need = lb.lowbit_lora_workspace_bytes(50, 3, 16, 96, 1040, torch.float16)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    rows, offsets = plan(t)
    d = {k: v.to(DEV) for k, v in t.items() if torch.is_tensor(v)}
    torch.cuda.synchronize()
    y = lb.lowbit_lora(d["x"], d["a"], d["b"], d["scales"], rows, offsets, d["base"], workspace=ws[:need], stream=s)
    s.synchronize()
    assert torch.equal(y, want) and (ws[need:] == 255).all()


@pytest.mark.parametrize("kind", ["lowbit", "f8", "linear"])
def test_module_beside_each_linear(kind):
    """base(x), then the batch's adapters; adapters of smaller rank; no plan, no adapters; compiled."""
    torch.manual_seed(4)
    K, N, M, L = 128, 72, 20, 3
    lin = torch.nn.Linear(K, N).to(DEV).half()
    linear = {"lowbit": lambda: lnn.LowbitLinear.from_linear(lin, 4, 32), "f8": lambda: lnn.F8Linear.from_linear(lin),
              "linear": lambda: lin}[kind]()
    m = lnn.LoraLinear(linear, L, 16)
    assert m.a.dtype == torch.float16 and m.a.device == DEV
    ids = torch.randint(-1, L, (4, 5), device=DEV)
    A, B = torch.randn(L, 8, K, device=DEV) / 11, torch.randn(L, N, 8, device=DEV) / 5
    for i in range(L):
        m.set_adapter(i, A[i], B[i], 0.5 + i)
    x = torch.randn(4, 5, K, device=DEV).half()
    with torch.no_grad():
        y0, y = m(x), m(x, lnn.adapter_plan(ids, L))
        assert torch.equal(y0, linear(x)) and y.shape == (4, 5, N)
        ref = f64(y0)
        for i in range(4):
            for j in range(5):
                e = ids[i, j].item()
                if e >= 0:
                    ref[i, j] += (0.5 + e) * (f64(B[e].half()) @ (f64(A[e].half()) @ f64(x[i, j])))
        # (the sums' own errors are far below half a step of fp16 at these sizes: 1.5 half steps)
        assert np.all(np.abs(f64(y) - ref) <= 1.5 * 2.0 ** -11 * (np.abs(ref) + 2.0 ** -3))
        fn = torch.compile(lambda x, p: m(x, p), fullgraph=True, backend="aot_eager")
        assert torch.equal(fn(x, lnn.adapter_plan(ids, L)), y)
