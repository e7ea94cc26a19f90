"""The operators around the experts and the adapters without a GPU: argument validation of the C ABI
(before any HIP call), the binding's checks, and the torch layer's shape functions and modules on the
meta device."""
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn

OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, 1, 2, 3, 6
F32, F16, BF16 = 0, 1, 2
A = 0x10000          # a fake, 256-byte aligned "device" address: never dereferenced
META = torch.device("meta")


# ------------------------------------------------------------------- C ABI --

@pytest.mark.parametrize("kw, status", [
    (dict(dt=3), UNSUPPORTED), (dict(score=2), UNSUPPORTED), (dict(T=-1), INVALID), (dict(T=(1 << 30) + 1), INVALID),
    (dict(T=(1 << 25) + 1), INVALID),        # more rows than a launch has blocks of four for
    (dict(E=0), INVALID), (dict(E=1025), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(E=16, groups=4, k=17), INVALID), (dict(groups=0), INVALID), (dict(groups=5), INVALID),
    (dict(E=130, groups=65), INVALID), (dict(kg=0), INVALID), (dict(kg=9), INVALID), (dict(best=0), INVALID),
    (dict(best=3), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(l=None), INVALID), (dict(e=None), INVALID), (dict(w=None), INVALID), (dict(l=A + 1), MISALIGNED),
    (dict(dt=F32, l=A + 2), MISALIGNED), (dict(b=A + 2), MISALIGNED), (dict(e=A + 2), MISALIGNED),
    (dict(w=A + 1), MISALIGNED), (dict(T=0), OK), (dict(T=0, l=None, e=None, w=None), OK),
])
def test_route_validation(lowbit_lib, kw, status):
    a = dict(l=A, dt=BF16, b=A, T=4, E=256, k=8, score=1, groups=8, kg=4, best=2, renorm=1, scale=1.0, e=A, w=A)
    a.update(kw)
    assert lowbit_lib.lowbit_moe_route(a["l"], a["dt"], a["b"], a["T"], a["E"], a["k"], a["score"], a["groups"],
                                       a["kg"], a["best"], a["renorm"], a["scale"], a["e"], a["w"], None) == status
    assert (lb.lowbit_last_error() == "") == (status == OK)


@pytest.mark.parametrize("kw, status", [
    (dict(bytes=2), UNSUPPORTED), (dict(bytes=0), UNSUPPORTED), (dict(T=-1), INVALID), (dict(k=0), INVALID),
    (dict(T=1 << 20, k=(1 << 10) + 1), INVALID), (dict(T=(1 << 30) + 1, k=1), INVALID), (dict(E=0), INVALID),
    (dict(E=(1 << 16) + 1), INVALID), (dict(ids=None), INVALID), (dict(rows=None), INVALID), (dict(off=None), INVALID),
    (dict(ids=A + 2), MISALIGNED), (dict(bytes=8, ids=A + 4), MISALIGNED), (dict(rows=A + 2), MISALIGNED),
    (dict(off=A + 1), MISALIGNED), (dict(pos=A + 2), MISALIGNED), (dict(T=0, off=None), INVALID),
    (dict(wb=256), WORKSPACE), (dict(ws=A + 64, wb=256), WORKSPACE),
])
def test_group_rows_validation(lowbit_lib, kw, status):
    a = dict(ids=A, bytes=4, T=4, k=2, E=8, rows=A, off=A, pos=A, ws=None, wb=0)
    a.update(kw)
    assert lowbit_lib.lowbit_group_rows(a["ids"], a["bytes"], a["T"], a["k"], a["E"], a["rows"], a["off"], a["pos"],
                                        a["ws"], a["wb"], None) == status
    assert lb.lowbit_last_error() != ""


@pytest.mark.parametrize("kw, status", [
    (dict(dt=3), UNSUPPORTED), (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(k=0), INVALID),
    (dict(k=(1 << 16) + 1), INVALID), (dict(N=0), INVALID), (dict(N=(1 << 30) + 1), INVALID),
    (dict(T=(1 << 30) + 1), INVALID), (dict(y=None), INVALID), (dict(pos=None), INVALID), (dict(w=None), INVALID),
    (dict(out=None), INVALID), (dict(y=A + 1), MISALIGNED), (dict(res=A + 1), MISALIGNED), (dict(out=A + 1), MISALIGNED),
    (dict(pos=A + 2), MISALIGNED), (dict(w=A + 2), MISALIGNED), (dict(T=0), OK),
    (dict(T=0, y=None, pos=None, w=None, out=None), OK),
])
def test_combine_validation(lowbit_lib, kw, status):
    a = dict(y=A, pos=A, w=A, res=A, out=A, dt=BF16, R=8, T=4, k=2, N=64)
    a.update(kw)
    assert lowbit_lib.lowbit_moe_combine(a["y"], a["pos"], a["w"], a["res"], a["out"], a["dt"], a["R"], a["T"], a["k"],
                                         a["N"], None) == status
    assert (lb.lowbit_last_error() == "") == (status == OK)


@pytest.mark.parametrize("kw, status", [
    (dict(dt=3), UNSUPPORTED), (dict(M=-1), INVALID), (dict(T=-1), INVALID), (dict(L=0), INVALID),
    (dict(L=(1 << 16) + 1), INVALID), (dict(rank=0), INVALID), (dict(rank=12), INVALID), (dict(rank=264), INVALID),
    (dict(N=0), INVALID), (dict(N=(1 << 23) + 1), INVALID), (dict(K=0), INVALID), (dict(K=40), INVALID),
    (dict(K=(1 << 23) + 16), INVALID), (dict(M=1 << 24, T=1 << 24, N=4096), INVALID), (dict(rows=None, T=5), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(off=None), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(x=A + 8), MISALIGNED), (dict(a=A + 8), MISALIGNED), (dict(b=A + 8), MISALIGNED),
    (dict(s=A + 2), MISALIGNED), (dict(rows=A + 2), MISALIGNED), (dict(off=A + 2), MISALIGNED),
    (dict(base=A + 1), MISALIGNED), (dict(y=A + 1), MISALIGNED), (dict(ws=None, wb=256), WORKSPACE),
    (dict(ws=A + 128), WORKSPACE), (dict(M=4000, T=4000, K=4096, wb=1024), WORKSPACE), (dict(T=0), OK),
    (dict(M=0, T=0, x=None, y=None, base=None, rows=None), OK), (dict(M=0), OK),
])
def test_lora_validation(lowbit_lib, kw, status):
    a = dict(x=A, a=A, b=A, s=A, rows=A, off=A, base=A, y=A, dt=BF16, M=4, T=4, L=3, rank=16, N=64, K=64, ws=A,
             wb=1 << 30)
    a.update(kw)
    assert lowbit_lib.lowbit_lora(a["x"], a["a"], a["b"], a["s"], a["rows"], a["off"], a["base"], a["y"], a["dt"],
                                  a["M"], a["T"], a["L"], a["rank"], a["N"], a["K"], a["ws"], a["wb"],
                                  None) == status
    assert (lb.lowbit_last_error() == "") == (status == OK)


@pytest.mark.parametrize("bad", [dict(T=0), dict(L=0), dict(rank=12), dict(N=0), dict(K=8), dict(T=-1)])
def test_lora_workspace_of_no_call(lowbit_lib, bad):
    a = dict(T=4000, L=3, rank=16, N=64, K=4096)
    assert lb.lowbit_lora_workspace_bytes(**a, dtype=torch.float16) > 0
    a.update(bad)
    assert lb.lowbit_lora_workspace_bytes(**a, dtype=torch.float16) == 0


# ----------------------------------------------------------------- binding --

def e(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype)


I32 = torch.int32
BF = torch.bfloat16


@pytest.mark.parametrize("args, kw, match", [
    ((e(4), 2), {}, "2-D"), ((e(4, 8, dtype=torch.float64), 2), {}, "not float32"), ((e(4, 8), 9), {}, "topk"),
    ((e(4, 8), 0), {}, "topk"), ((e(4, 8), 2), dict(bias=e(7)), "bias"), ((e(4, 8), 2), dict(bias=e(8, dtype=BF)), "bias"),
    ((e(4, 8), 2), dict(experts=e(4, 2)), "experts"), ((e(4, 8), 2), dict(weights=e(4, 3)), "weights"),
    ((e(4, 8), 2), {}, "GPU memory"),
])
def test_route_refuses(lowbit_lib, args, kw, match):
    with pytest.raises(ValueError, match=match):
        lb.lowbit_moe_route(*args, **kw)


@pytest.mark.parametrize("args, kw, match", [
    ((e(4, dtype=I32), 8), {}, "2-D"), ((e(4, 0, dtype=I32), 8), {}, "2-D"), ((e(4, 2), 8), {}, "int32 or int64"),
    ((e(4, 2, dtype=I32), 0), {}, "E=0"), ((e(4, 2, dtype=I32), 1 << 17), {}, "E="),
    ((e(4, 2, dtype=I32), 8), dict(rows=e(7, dtype=I32)), "rows"), ((e(4, 2, dtype=I32), 8), dict(offsets=e(8, dtype=I32)), "offsets"),
    ((e(4, 2, dtype=I32), 8), dict(position=e(8, dtype=I32)), "position"), ((e(4, 2, dtype=I32), 8), {}, "GPU memory"),
])
def test_group_rows_refuses(lowbit_lib, args, kw, match):
    with pytest.raises(ValueError, match=match):
        lb.lowbit_group_rows(*args, **kw)


@pytest.mark.parametrize("args, kw, match", [
    ((e(4), e(2, 2, dtype=I32), e(2, 2)), {}, "must be"), ((e(4, 8), e(4, dtype=I32), e(2, 2)), {}, "must be"),
    ((e(4, 8, dtype=torch.float64), e(2, 2, dtype=I32), e(2, 2)), {}, "not float32"),
    ((e(4, 8), e(2, 2, dtype=torch.int64), e(2, 2)), {}, "position"), ((e(4, 8), e(2, 2, dtype=I32), e(2, 2, dtype=BF)), {}, "weights"),
    ((e(4, 8), e(2, 2, dtype=I32), e(2, 3)), {}, "weights"),
    ((e(4, 8), e(2, 2, dtype=I32), e(2, 2)), dict(residual=e(4, 8)), "residual"),
    ((e(4, 8), e(2, 2, dtype=I32), e(2, 2)), dict(out=e(2, 8, dtype=BF)), "out"),
    ((e(4, 8), e(2, 2, dtype=I32), e(2, 2)), {}, "GPU memory"),
])
def test_combine_refuses(lowbit_lib, args, kw, match):
    with pytest.raises(ValueError, match=match):
        lb.lowbit_moe_combine(*args, **kw)


@pytest.mark.parametrize("kw, match", [
    (dict(x=e(4)), "must be"), (dict(a=e(32, 8)), "must be"), (dict(b=e(3, 40, 8, 1)), "must be"),
    (dict(x=e(4, 32, dtype=torch.float64)), "not float32"), (dict(a=e(3, 8, 48)), "a must"), (dict(a=e(3, 8, 32, dtype=BF)), "a must"),
    (dict(b=e(2, 40, 8)), "b must"), (dict(b=e(3, 40, 16)), "b must"), (dict(offsets=e(3, dtype=I32)), "offsets"),
    (dict(offsets=e(4, dtype=torch.int64)), "offsets"), (dict(scales=e(4)), "scales"), (dict(scales=e(3, dtype=BF)), "scales"),
    (dict(rows=e(4, 1, dtype=I32)), "rows"), (dict(rows=e(4, dtype=torch.int64)), "rows"), (dict(base=e(4, 41)), "base"),
    (dict(y=e(3, 40)), "y must"), (dict(workspace=e(4096)), "workspace"), (dict(), "GPU memory"),
])
def test_lora_refuses(lowbit_lib, kw, match):
    a = dict(x=e(4, 32), a=e(3, 8, 32), b=e(3, 40, 8), scales=e(3), rows=e(4, dtype=I32), offsets=e(4, dtype=I32),
             base=e(4, 40))
    a.update(kw)
    with pytest.raises(ValueError, match=match):
        lb.lowbit_lora(**a)


def test_signatures_are_declared(lowbit_lib):
    for name, n in (("lowbit_moe_route", 15), ("lowbit_group_rows", 11), ("lowbit_moe_combine", 11), ("lowbit_lora", 18),
                    ("lowbit_lora_workspace_bytes", 6), ("lowbit_group_rows_workspace_bytes", 3)):
        assert len(getattr(lowbit_lib, name).argtypes) == n


def test_calls_run_with_the_tensors_device_current(lowbit_lib, monkeypatch):
    """Tensors on GPU 1 while GPU 0 is current: schedules and launches are those of GPU 1."""
    current, seen = [0], []

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(lb, "_entry", lambda name: (None, lambda *args: (seen.append((name, current[0])), 0)[1]))
    monkeypatch.setattr(lb, "_placed", lambda *tensors: 1)
    monkeypatch.setattr(lb, "_stream_of", lambda index, stream: 0)
    lb.lowbit_moe_route(e(3, 8), 2)
    lb.lowbit_group_rows(e(3, 2, dtype=I32), 8)
    lb.lowbit_moe_combine(e(6, 8), e(3, 2, dtype=I32), e(3, 2))
    lb.lowbit_lora(e(4, 32), e(3, 8, 32), e(3, 40, 8), None, None, e(4, dtype=I32), None)
    assert seen == [("lowbit_moe_route", 1), ("lowbit_group_rows", 1), ("lowbit_moe_combine", 1),
                    ("lowbit_lora_workspace_bytes", 1), ("lowbit_lora", 1)]


# ------------------------------------------------------------- torch layer --

def m(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device=META)


def test_shape_functions():
    ex, w = torch.ops.lowbit.moe_route(m(2, 7, 24, dtype=BF), m(24), 3, 1, 4, 2, 2, True, 1.0)
    assert ex.shape == w.shape == (2, 7, 3) and ex.dtype == I32 and w.dtype == torch.float32
    rows, offsets, position = torch.ops.lowbit.group_rows(m(14, 3, dtype=I32), 24)
    assert rows.shape == (42,) and offsets.shape == (25,) and position.shape == (14, 3)
    assert {rows.dtype, offsets.dtype, position.dtype} == {I32}
    out = torch.ops.lowbit.moe_combine(m(42, 40, dtype=BF), position, m(14, 3), m(14, 40, dtype=BF))
    assert out.shape == (14, 40) and out.dtype == BF
    y = torch.ops.lowbit.lora(m(2, 5, 32, dtype=BF), m(3, 8, 32, dtype=BF), m(3, 40, 8, dtype=BF), m(3),
                              m(10, dtype=I32), m(4, dtype=I32), m(2, 5, 40, dtype=BF))
    assert y.shape == (2, 5, 40) and y.dtype == BF


@pytest.mark.parametrize("call", [
    lambda: torch.ops.lowbit.moe_route(m(4, 8, dtype=torch.float64), None, 2, 0, 1, 1, 1, True, 1.0),
    lambda: torch.ops.lowbit.moe_route(m(4, 2000), None, 2, 0, 1, 1, 1, True, 1.0),
    lambda: torch.ops.lowbit.moe_route(m(4, 8), None, 9, 0, 1, 1, 1, True, 1.0),
    lambda: torch.ops.lowbit.moe_route(m(4, 8), None, 2, 2, 1, 1, 1, True, 1.0),
    lambda: torch.ops.lowbit.moe_route(m(4, 8), None, 2, 0, 3, 1, 1, True, 1.0),
    lambda: torch.ops.lowbit.moe_route(m(4, 8), None, 2, 0, 2, 3, 1, True, 1.0),
    lambda: torch.ops.lowbit.moe_route(m(4, 8), None, 2, 0, 2, 1, 3, True, 1.0),
    lambda: torch.ops.lowbit.moe_route(m(4, 8), m(8, dtype=BF), 2, 0, 1, 1, 1, True, 1.0),
    lambda: torch.ops.lowbit.group_rows(m(4, 2), 8),
    lambda: torch.ops.lowbit.group_rows(m(4, dtype=I32), 8),
    lambda: torch.ops.lowbit.group_rows(m(4, 2, dtype=I32), 0),
    lambda: torch.ops.lowbit.moe_combine(m(4, 8), m(2, 2), m(2, 2), None),
    lambda: torch.ops.lowbit.moe_combine(m(4, 8), m(2, 2, dtype=I32), m(2, 2, dtype=BF), None),
    lambda: torch.ops.lowbit.moe_combine(m(4, 8), m(2, 2, dtype=I32), m(2, 2), m(2, 9)),
    lambda: torch.ops.lowbit.lora(m(4, 40), m(3, 8, 40), m(3, 40, 8), None, None, m(4, dtype=I32), None),
    lambda: torch.ops.lowbit.lora(m(4, 32), m(3, 12, 32), m(3, 40, 12), None, None, m(4, dtype=I32), None),
    lambda: torch.ops.lowbit.lora(m(4, 32), m(3, 264, 32), m(3, 40, 264), None, None, m(4, dtype=I32), None),
    lambda: torch.ops.lowbit.lora(m(4, 32), m(3, 8, 32), m(2, 40, 8), None, None, m(4, dtype=I32), None),
    lambda: torch.ops.lowbit.lora(m(4, 32), m(3, 8, 32), m(3, 40, 8), None, None, m(3, dtype=I32), None),
    lambda: torch.ops.lowbit.lora(m(4, 32), m(3, 8, 32), m(3, 40, 8), None, None, m(4, dtype=I32), m(4, 41)),
])
def test_shape_functions_refuse(call):
    with pytest.raises(ValueError):
        call()


def test_modules_on_meta():
    r = lnn.MoeRouter(24, 3, "sigmoid", bias=True, groups=4, topk_groups=2, device=META)
    ex, w = r.half()(m(5, 24))
    assert ex.shape == (5, 3) and r.bias.dtype == torch.float32
    experts = lnn.F8Experts(24, 64, 48, device=META)
    assert experts(m(5, 64, dtype=BF), ex, w).shape == (5, 64)
    for linear in (lnn.F8Linear(64, 40, device=META), lnn.LowbitLinear(64, 40, 4, 32, dtype=BF, device=META),
                   torch.nn.Linear(64, 40, device=META, dtype=BF)):
        lora = lnn.LoraLinear(linear, 3, 8)
        assert lora.a.dtype == BF and lora.a.device == META
        lora = lora.half()
        assert lora.a.dtype == lora.b.dtype == torch.float16 and lora.scales.dtype == torch.float32
        if not isinstance(linear, lnn.LowbitLinear):       # (its type is that of its scales at the start)
            y = lora(m(2, 3, 64, dtype=torch.float16), lnn.adapter_plan(m(2, 3, dtype=torch.int16), 3))
            assert y.shape == (2, 3, 40) and y.dtype == torch.float16


@pytest.mark.parametrize("make", [
    lambda: lnn.MoeRouter(8, 9), lambda: lnn.MoeRouter(8, 2, "tanh"), lambda: lnn.MoeRouter(8, 2, groups=3),
    lambda: lnn.MoeRouter(8, 2)(m(4, 9)),
    lambda: lnn.LoraLinear(torch.nn.Linear(64, 40, device=META), 0, 8),
    lambda: lnn.LoraLinear(torch.nn.Linear(64, 40, device=META), 2, 12),
    lambda: lnn.LoraLinear(torch.nn.Linear(72, 40, device=META), 2, 8),
    lambda: lnn.LoraLinear(torch.nn.Linear(64, 40, device=META, dtype=torch.float64), 2, 8),
    lambda: lnn.LoraLinear(torch.nn.Linear(64, 40), 2, 8).set_adapter(2, e(8, 64), e(40, 8)),
    lambda: lnn.LoraLinear(torch.nn.Linear(64, 40), 2, 8).set_adapter(0, e(16, 64), e(40, 16)),
    lambda: lnn.LoraLinear(torch.nn.Linear(64, 40), 2, 8).set_adapter(0, e(8, 64), e(40, 4)),
])
def test_modules_reject(make):
    with pytest.raises(ValueError):
        make()


def test_set_adapter_fills_up_with_zeros():
    lora = lnn.LoraLinear(torch.nn.Linear(16, 5), 2, 8)
    lora.a.fill_(7.0)
    lora.b.fill_(7.0)
    lora.set_adapter(1, torch.ones(3, 16), torch.ones(5, 3), 0.25)
    assert (lora.a[1, :3] == 1).all() and (lora.a[1, 3:] == 0).all() and (lora.b[1, :, 3:] == 0).all()
    assert (lora.a[0] == 7).all() and lora.scales.tolist() == [1.0, 0.25]
