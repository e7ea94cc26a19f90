"""The 8-bit path without a GPU: argument validation of the C ABI (before any HIP call), the
binding's checks, and the torch layer's shape functions and modules on the meta device."""
import ctypes

import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 6
F32, F16, BF16 = 0, 1, 2
A = 0x10000          # a fake, 256-byte aligned "device" address: never dereferenced
F8 = torch.float8_e4m3fn
META = torch.device("meta")


# ------------------------------------------------------------------ C ABI --

def norm(lib, **kw):
    a = dict(x=A, residual=A, weight=A, eps=1e-5, dt=BF16, M=4, K=256, fmt=2, q=A, qs=A, sum=A, y=None)
    a.update(kw)
    return lib.lowbit_add_rmsnorm_q8(a["x"], a["residual"], a["weight"], a["eps"], a["dt"], a["M"], a["K"],
                                     a["fmt"], a["q"], a["qs"], a["sum"], a["y"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(dt=3), UNSUPPORTED), (dict(fmt=3), UNSUPPORTED), (dict(fmt=-1), UNSUPPORTED),
    (dict(K=0), INVALID), (dict(K=40), INVALID), (dict(K=48, fmt=1), INVALID),
    (dict(K=(1 << 23) + 16), INVALID), (dict(M=-1), INVALID), (dict(M=1 << 22), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=2.0), INVALID), (dict(x=None), INVALID), (dict(sum=None), INVALID),
    (dict(residual=None), INVALID), (dict(q=None), INVALID), (dict(qs=None), INVALID),
    (dict(fmt=0), INVALID), (dict(fmt=0, q=None, qs=None), INVALID), (dict(x=A + 8), MISALIGNED),
    (dict(residual=A + 8), MISALIGNED), (dict(weight=A + 8), MISALIGNED), (dict(sum=A + 8), MISALIGNED),
    (dict(y=A + 8), MISALIGNED), (dict(q=A + 8), MISALIGNED), (dict(qs=A + 2), MISALIGNED),
    (dict(M=0), OK), (dict(M=0, x=None, residual=None, sum=None, q=None, qs=None), OK),
])
def test_norm_validation(lowbit_lib, kw, status):
    assert norm(lowbit_lib, **kw) == status
    assert (lb.lowbit_last_error() == "") == (status == OK)


@pytest.mark.parametrize("kw, status", [
    (dict(dt=3), UNSUPPORTED), (dict(M=-1), INVALID), (dict(K=24), INVALID), (dict(K=0), INVALID),
    (dict(M=1 << 28), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(x=A + 8), MISALIGNED), (dict(q=A + 4), MISALIGNED), (dict(s=A + 1), MISALIGNED), (dict(M=0), OK),
])
def test_quantize_act_f8_validation(lowbit_lib, kw, status):
    a = dict(x=A, dt=BF16, M=4, K=256, q=A, s=A)
    a.update(kw)
    assert lowbit_lib.lowbit_quantize_act_f8(a["x"], a["dt"], a["M"], a["K"], a["q"], a["s"], None) == status


@pytest.mark.parametrize("kw, status", [
    (dict(dt=3), UNSUPPORTED), (dict(E=0), INVALID), (dict(E=(1 << 16) + 1), INVALID), (dict(N=0), INVALID),
    (dict(K=24), INVALID), (dict(N=1 << 30, K=1 << 20), INVALID), (dict(w=None), INVALID),
    (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(w=A + 8), MISALIGNED),
    (dict(q=A + 4), MISALIGNED), (dict(s=A + 2), MISALIGNED),
])
def test_quantize_weight_f8_validation(lowbit_lib, kw, status):
    a = dict(w=A, dt=F32, E=1, N=64, K=256, q=A, s=A)
    a.update(kw)
    assert lowbit_lib.lowbit_quantize_weight_f8(a["w"], a["dt"], a["E"], a["N"], a["K"], a["q"], a["s"],
                                                None) == status


LINEAR_CASES = [
    (dict(dt=5), UNSUPPORTED), (dict(K=0), INVALID), (dict(K=40), INVALID), (dict(N=0), INVALID),
    (dict(K=(1 << 23) + 16), INVALID), (dict(N=(1 << 30) + 1), INVALID), (dict(xq=None), INVALID),
    (dict(xs=None), INVALID), (dict(wq=None), INVALID), (dict(ws=None), INVALID), (dict(y=None), INVALID),
    (dict(xq=A + 8), MISALIGNED), (dict(wq=A + 8), MISALIGNED), (dict(xs=A + 2), MISALIGNED),
    (dict(ws=A + 2), MISALIGNED), (dict(y=A + 1), MISALIGNED), (dict(bias=A + 1), MISALIGNED),
    (dict(wkb=64), WORKSPACE), (dict(wk=A + 16, wkb=64), WORKSPACE),
]


@pytest.mark.parametrize("kw, status", LINEAR_CASES + [
    (dict(M=-1), INVALID), (dict(M=(1 << 30) + 1), INVALID), (dict(M=0), OK),
    (dict(M=0, xq=None, xs=None, y=None), OK), (dict(M=0, wq=None), INVALID)])
def test_linear_f8_validation(lowbit_lib, kw, status):
    a = dict(xq=A, xs=A, wq=A, ws=A, bias=None, y=A, dt=BF16, M=4, N=64, K=256, wk=None, wkb=0)
    a.update(kw)
    st = lowbit_lib.lowbit_linear_f8(a["xq"], a["xs"], a["wq"], a["ws"], a["bias"], a["y"], a["dt"], a["M"],
                                     a["N"], a["K"], a["wk"], a["wkb"], None)
    assert st == status
    assert (lb.lowbit_last_error() == "") == (status == OK)


@pytest.mark.parametrize("kw, status", LINEAR_CASES + [
    (dict(off=None), INVALID), (dict(E=0), INVALID), (dict(E=(1 << 16) + 1), INVALID),
    (dict(M=5), INVALID), (dict(T=-1, M=-1), INVALID), (dict(rows=A, M=0), INVALID),
    (dict(rows=A + 2), MISALIGNED), (dict(off=A + 2), MISALIGNED), (dict(rows=A, M=9, dt=7), UNSUPPORTED),
    (dict(T=0, M=0), OK), (dict(T=0, M=7, rows=A), OK)])
def test_linear_f8_grouped_validation(lowbit_lib, kw, status):
    a = dict(xq=A, xs=A, rows=None, off=A, wq=A, ws=A, bias=None, y=A, dt=BF16, M=4, T=4, E=2, N=64, K=256,
             wk=None, wkb=0)
    a.update(kw)
    st = lowbit_lib.lowbit_linear_f8_grouped(a["xq"], a["xs"], a["rows"], a["off"], a["wq"], a["ws"],
                                             a["bias"], a["y"], a["dt"], a["M"], a["T"], a["E"], a["N"],
                                             a["K"], a["wk"], a["wkb"], None)
    assert st == status


@pytest.mark.parametrize("M, T, E, N, K, dtype, splits", [
    (1, 1, 0, 14336, 4096, "bf16", 0),        # few rows: no workspace
    (64, 64, 0, 4096, 14336, "bf16", 4),      # tiles of 64 columns
    (128, 128, 0, 4096, 14336, "f32", 4),
    (20, 20, 0, 4096, 4096, "f16", 0),
    (8192, 8192, 0, 14336, 4096, "bf16", 0),  # 256 x 256: none
    (64, 64, 0, 4098, 14336, "bf16", 5),      # planes padded to a multiple of 4 columns
    (30, 60, 2, 1024, 8192, "bf16", 6),       # grouped: planes of T rows
    (4, 0, 2, 64, 256, "bf16", 0), (4, 4, 0, 64, 40, "bf16", 0),
])
def test_workspace_bytes(lowbit_lib, M, T, E, N, K, dtype, splits):
    """The schedule on a 256-CU device, seen through its fp32 planes of T x N."""
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    assert lb.lowbit_linear_f8_workspace_bytes(M, T, E, N, K, dt) == splits * T * -(-N // 4) * 4 * 4


def test_signatures_are_declared(lowbit_lib):
    """ctypes passes eps as a C float and the sizes as 64-bit integers."""
    assert lowbit_lib.lowbit_add_rmsnorm_q8.argtypes[3] is ctypes.c_float
    assert lowbit_lib.lowbit_linear_f8_grouped.argtypes[9:14] == [ctypes.c_int64] * 5


# ---------------------------------------------------------------- binding --

M, N, K, E, T = 3, 40, 272, 4, 6


def f8_args(**kw):
    a = dict(xq=torch.zeros(M, K, dtype=F8), xs=torch.zeros(M, 3), wq=torch.zeros(N, K, dtype=F8),
             ws=torch.zeros(1, 3), bias=None, dtype=torch.bfloat16, y=None)
    a.update(kw)
    return lb.lowbit_linear_f8(a["xq"], a["xs"], a["wq"], a["ws"], a["bias"], a["dtype"], y=a["y"])


def test_linear_f8_reaches_the_device_check(lowbit_lib):
    with pytest.raises(ValueError, match="GPU memory"):
        f8_args()


@pytest.mark.parametrize("kw, match", [
    (dict(xq=torch.zeros(M, K)), "xq must be"), (dict(xq=torch.zeros(K, dtype=F8)), "xq must be"),
    (dict(xs=torch.zeros(M, 2)), "xscale must be"), (dict(xs=torch.zeros(M, 3).half()), "xscale must be"),
    (dict(wq=torch.zeros(N, 256, dtype=F8)), "wq must be"), (dict(wq=torch.zeros(N, K)), "wq must be"),
    (dict(ws=torch.zeros(2, 3)), "wscale must be"), (dict(bias=torch.zeros(N)), "bias must be"),
    (dict(bias=torch.zeros(N - 1, dtype=torch.bfloat16)), "bias must be"),
    (dict(y=torch.zeros(M, N)), "y must be"), (dict(dtype=torch.float64), "dtype"),
    (dict(y=torch.zeros(M, N + 1, dtype=torch.bfloat16)), "y must be"),
])
def test_linear_f8_refuses(lowbit_lib, kw, match):
    with pytest.raises(ValueError, match=match):
        f8_args(**kw)


def grouped_args(**kw):
    a = dict(xq=torch.zeros(M, K, dtype=F8), xs=torch.zeros(M, 3),
             off=torch.zeros(E + 1, dtype=torch.int32), wq=torch.zeros(E, N, K, dtype=F8),
             ws=torch.zeros(E, 1, 3), bias=None, dtype=torch.float16,
             rows=torch.zeros(T, dtype=torch.int32), y=None)
    a.update(kw)
    return lb.lowbit_linear_f8_grouped(a["xq"], a["xs"], a["off"], a["wq"], a["ws"], a["bias"], a["dtype"],
                                       rows=a["rows"], y=a["y"])


@pytest.mark.parametrize("kw, match", [
    ({}, "GPU memory"), (dict(rows=None), "GPU memory"),
    (dict(off=torch.zeros(E, dtype=torch.int32)), "offsets must be"),
    (dict(off=torch.zeros(E + 1, dtype=torch.int64)), "offsets must be"),
    (dict(rows=torch.zeros(T, dtype=torch.int64)), "rows must be"),
    (dict(rows=torch.zeros(T, 1, dtype=torch.int32)), "rows must be"),
    (dict(wq=torch.zeros(N, K, dtype=F8)), "wq"), (dict(ws=torch.zeros(E, 3)), "wscale must be"),
    (dict(y=torch.zeros(M, N, dtype=torch.float16)), "y must be"),
    (dict(bias=torch.zeros(N, dtype=torch.float16)), "bias must be"),
])
def test_grouped_refuses(lowbit_lib, kw, match):
    with pytest.raises(ValueError, match=match):
        grouped_args(**kw)


def norm_args(**kw):
    a = dict(x=torch.zeros(M, K, dtype=torch.bfloat16), weight=None, fmt=lb.Q8_F8)
    a.update(kw)
    x, w, fmt = a.pop("x"), a.pop("weight"), a.pop("fmt")
    return lb.lowbit_add_rmsnorm_q8(x, w, 1e-5, fmt, **a)


BF = torch.bfloat16


@pytest.mark.parametrize("kw, match", [
    ({}, "GPU memory"), (dict(residual=torch.zeros(M, K, dtype=BF)), "GPU memory"),
    (dict(x=torch.zeros(M, K, dtype=torch.float64)), "x dtype"), (dict(x=torch.zeros(K)), "x must be 2-D"),
    (dict(weight=torch.zeros(K)), "weight must be"), (dict(weight=torch.zeros(K + 1, dtype=BF)), "weight must"),
    (dict(residual=torch.zeros(M, K)), "residual must be"), (dict(h=torch.zeros(M, K, dtype=BF)), "h is the"),
    (dict(fmt=3), "fmt must be"), (dict(fmt=lb.Q8_NONE, q=torch.zeros(M, K, dtype=F8)), "no meaning"),
    (dict(q=torch.zeros(M, K, dtype=torch.int8)), "q must be"), (dict(qscale=torch.zeros(M)), "qscale must be"),
    (dict(fmt=lb.Q8_I8, qscale=torch.zeros(M, 3)), "qscale must be"),
    (dict(y=torch.zeros(M, K)), "y must be"),
    (dict(residual=torch.zeros(M, K, dtype=BF), h=torch.zeros(M, K)), "h must be"),
    (dict(x=torch.zeros(K, M, dtype=BF).t()), "GPU memory"),
])
def test_norm_refuses(lowbit_lib, kw, match):
    with pytest.raises(ValueError, match=match):
        norm_args(**kw)


# ------------------------------------------------------------ torch layer --

@pytest.mark.parametrize("lead", [(), (5,), (2, 3)])
@pytest.mark.parametrize("fmt", [lb.Q8_I8, lb.Q8_F8])
def test_norm_shape_functions(lead, fmt):
    x = torch.empty((*lead, 288), dtype=BF, device=META)
    w = torch.empty(288, dtype=BF, device=META)
    spans = lead if fmt == lb.Q8_I8 else (*lead, 3)
    code = torch.int8 if fmt == lb.Q8_I8 else F8
    for q, s, *h in (torch.ops.lowbit.rmsnorm_q8(x, w, 1e-6, fmt),
                     torch.ops.lowbit.add_rmsnorm_q8(x, x, None, 1e-6, fmt)):
        assert q.shape == x.shape and q.dtype == code and s.shape == spans and s.dtype == torch.float32
        assert all(t.shape == x.shape and t.dtype == BF for t in h)
    for bad in (lambda: torch.ops.lowbit.rmsnorm_q8(x, w, 1e-6, 0),
                lambda: torch.ops.lowbit.rmsnorm_q8(x[..., :24], None, 1e-6, fmt),
                lambda: torch.ops.lowbit.rmsnorm_q8(x, w.float(), 1e-6, fmt),
                lambda: torch.ops.lowbit.add_rmsnorm_q8(x, x.float(), w, 1e-6, fmt)):
        with pytest.raises(Exception):
            bad()


def test_linear_shape_functions():
    x = torch.empty((2, 5, 272), dtype=BF, device=META)
    xq, xs = torch.ops.lowbit.quantize_act_f8(x)
    wq, ws = torch.ops.lowbit.quantize_weight_f8(torch.empty((200, 272), device=META))
    assert wq.shape == (200, 272) and wq.dtype == F8 and ws.shape == (2, 3)
    y = torch.ops.lowbit.linear_f8(xq, xs, wq, ws, None, BF)
    assert y.shape == (2, 5, 200) and y.dtype == BF
    w3, s3 = torch.ops.lowbit.quantize_weight_f8(torch.empty((4, 200, 272), device=META))
    assert s3.shape == (4, 2, 3)
    off = torch.empty(5, dtype=torch.int32, device=META)
    rows = torch.empty(9, dtype=torch.int32, device=META)
    g = torch.ops.lowbit.linear_f8_grouped(xq[0], xs[0], rows, off, w3, s3, None, torch.float16)
    assert g.shape == (9, 200) and g.dtype == torch.float16
    with pytest.raises(Exception):
        torch.ops.lowbit.linear_f8(xq, xs, wq[:, :256], ws, None, BF)
    with pytest.raises(Exception):
        torch.ops.lowbit.linear_f8(xq, xs, wq, ws, torch.empty(200, device=META), BF)


def test_modules_on_meta():
    m = lnn.F8Linear(272, 200, dtype=BF, device=META)
    assert m(torch.empty((3, 272), dtype=BF, device=META)).shape == (3, 200)
    assert "in_features=272" in repr(m)
    with pytest.raises(ValueError):
        lnn.F8Linear(40, 8)
    e = lnn.F8Experts(4, 64, 96, device=META)
    assert e.gate_up.shape == (4, 192, 64) and e.down_scale.shape == (4, 1, 1)
    with pytest.raises(ValueError):
        lnn.F8Experts(4, 60, 96)
    net = torch.nn.Sequential(torch.nn.Linear(64, 32, device=META), torch.nn.Linear(24, 8, device=META),
                              torch.nn.Sequential(torch.nn.Linear(32, 16, bias=False, device=META)))
    lnn.quantize_linears_f8(net, dtype=BF, filter_fn=lambda mod, name: name != "0")
    assert type(net[0]) is torch.nn.Linear and type(net[1]) is torch.nn.Linear
    assert type(net[2][0]) is lnn.F8Linear and net[2][0].bias is None
