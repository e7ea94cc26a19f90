"""The 8-bit path's limits and modules without a GPU."""
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
from bit_groupwise_weight_amd import nn as lnn

OK, INVALID = 0, 1
BF16 = 2


@pytest.mark.parametrize("M, K, within", [
    ((1 << 28) - 16, 16, True), ((1 << 28) - 15, 16, False), ((1 << 28) - 1, 128, False),
    ((1 << 27) - 8, 144, True), ((1 << 27) - 7, 144, False), ((1 << 12) - 1, 1 << 23, True), (1 << 12, 1 << 23, False),
])
def test_quantize_act_f8_takes_no_more_than_a_launch_can_hold(lowbit_lib, M, K, within):
    """16 threads a block of 128: 2^32 - 256 threads at most.  (The sizes are checked before the
    NULL pointers.)"""
    assert lowbit_lib.lowbit_quantize_act_f8(None, BF16, M, K, None, None, None) == INVALID
    assert ("NULL" in lb.lowbit_last_error()) == within
    assert ("2^28 - 16" in lb.lowbit_last_error()) != within


@pytest.mark.parametrize("M, T, E, N, K, splits", [
    (226200, 3841, 2, 2441, 19072, 2),       # a gathered xq past 4 GiB has no 256 x 256 tiles: K splits
    (99400, 803, 2, 10552, 43648, 4),
    (225000, 3841, 2, 2441, 19072, 0),       # just below: 256 x 256
])
def test_workspace_covers_the_schedule_of_gathered_rows(lowbit_lib, M, T, E, N, K, splits):
    """The schedule on a 256-CU device, seen through its fp32 planes of T x N."""
    need = lb.lowbit_linear_f8_workspace_bytes(M, T, E, N, K, torch.bfloat16)
    assert need == splits * T * -(-N // 4) * 4 * 4


def test_calls_and_workspace_queries_run_with_the_tensors_device_current(lowbit_lib, monkeypatch):
    """Tensors on GPU 1 while GPU 0 is current: schedules are the device's own, so the query that
    sizes the workspace and the call must both see GPU 1."""
    current, seen = [0], []

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    def entry(name):
        return None, lambda *args: (seen.append((name, current[0])), 0)[1]

    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(lb, "_entry", entry)
    monkeypatch.setattr(lb, "_placed", lambda *tensors: 1)
    monkeypatch.setattr(lb, "_stream_of", lambda index, stream: 0)
    f8 = torch.float8_e4m3fn
    xq, xs = torch.zeros(3, 256, dtype=f8), torch.zeros(3, 2)
    wq, ws = torch.zeros(2, 40, 256, dtype=f8), torch.zeros(2, 1, 2)
    lb.lowbit_linear_f8(xq, xs, wq[0], ws[0], None, torch.bfloat16)
    lb.lowbit_linear_f8_grouped(xq, xs, torch.zeros(3, dtype=torch.int32), wq, ws, None, torch.bfloat16)
    assert seen == [("lowbit_linear_f8_workspace_bytes", 1), ("lowbit_linear_f8", 1),
                    ("lowbit_linear_f8_workspace_bytes", 1), ("lowbit_linear_f8_grouped", 1)]


# ---------------------------------------------------------------- modules --

def f8_modules():
    lin = lnn.F8Linear(272, 200, dtype=torch.bfloat16)
    lin.wq.view(torch.uint8).random_(0, 120)
    lin.wscale.uniform_(1e-6, 1.0)
    exp = lnn.F8Experts(3, 64, 96)
    exp.down.view(torch.uint8).random_(0, 120)
    exp.down_scale.uniform_(1e-6, 1.0)
    return [lin, exp]


CASTS = [("half", lambda m: m.half(), torch.float16), ("to f16", lambda m: m.to(torch.float16), torch.float16),
         ("float", lambda m: m.float(), torch.float32), ("to cpu f32", lambda m: m.to("cpu", torch.float32), torch.float32),
         ("bfloat16", lambda m: m.bfloat16(), torch.bfloat16), ("type", lambda m: m.type(torch.float16), torch.float16),
         ("like", lambda m: m.to(torch.zeros(1, dtype=torch.float16)), torch.float16), ("cpu", lambda m: m.cpu(), torch.bfloat16)]


@pytest.mark.parametrize("name, cast, dtype", CASTS, ids=[c[0] for c in CASTS])
def test_a_cast_leaves_codes_and_scales(name, cast, dtype):
    """Codes and scales stay bit for bit; outputs and bias take the type."""
    for m in f8_modules():
        before = {n: b.clone() for n, b in m.named_buffers()}
        assert cast(torch.nn.Sequential(m))[0] is m and m.dtype == dtype
        for n, b in m.named_buffers():
            if n == "bias":
                assert b.dtype == dtype
            else:
                assert b.dtype == before[n].dtype
                assert torch.equal(b.view(torch.uint8), before[n].view(torch.uint8))


def test_a_cast_module_runs_on_meta():
    m = lnn.F8Linear(272, 200, dtype=torch.bfloat16).half().to("meta")
    assert m.wq.is_meta and m.wscale.is_meta and m.bias.is_meta
    y = m(torch.empty((3, 272), dtype=torch.float16, device="meta"))
    assert y.shape == (3, 200) and y.dtype == torch.float16
    m = lnn.F8Linear(272, 200, bias=False, device="meta").to("meta", torch.float32)
    assert m.wq.dtype == torch.float8_e4m3fn and m.wscale.dtype == torch.float32 and m.dtype == torch.float32
    assert m.to_empty(device="cpu").wq.device.type == "cpu"


@pytest.mark.parametrize("dtype", [torch.float64, torch.float8_e4m3fn])
def test_a_cast_to_a_type_without_outputs_is_refused(dtype):
    for m in f8_modules():
        before = {n: b.clone() for n, b in m.named_buffers()}
        with pytest.raises(ValueError, match="computes in one of"):
            m.to(dtype)
        assert m.dtype == torch.bfloat16
        for n, b in m.named_buffers():
            assert b.dtype == before[n].dtype and torch.equal(b.view(torch.uint8), before[n].view(torch.uint8))


def shared_model(device):
    lin, block = torch.nn.Linear(64, 64, device=device), torch.nn.Sequential(torch.nn.Linear(64, 32, device=device))
    return torch.nn.ModuleDict({"a": lin, "b": torch.nn.Sequential(lin, lin), "c": block, "d": block})


def test_a_shared_linear_stays_shared():
    """A layer at several places, and a block at two, become one quantized layer each."""
    net = lnn.quantize_linears_f8(shared_model("meta"))
    assert type(net["a"]) is lnn.F8Linear and net["b"][0] is net["a"] and net["b"][1] is net["a"]
    assert net["c"] is net["d"] and type(net["c"][0]) is lnn.F8Linear
    assert not any(isinstance(m, torch.nn.Linear) for m in net.modules())


def test_a_shared_linear_with_a_filter():
    """The filter sees every place; the layer stays where it excludes it."""
    names = []
    net = shared_model("meta")
    lin = net["a"]
    lnn.quantize_linears_f8(net, filter_fn=lambda m, name: names.append(name) or name != "b.1")
    assert names == ["a", "b.0", "b.1", "c.0", "d.0"]
    assert net["b"][0] is net["a"] is not lin and net["b"][1] is lin


# -------------------------------------------------------- shape functions --

F8, META = torch.float8_e4m3fn, "meta"


def empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=META)


@pytest.mark.parametrize("call", [
    lambda op: op.quantize_weight_f8(empty(8, 24)), lambda op: op.quantize_weight_f8(empty(8)),
    lambda op: op.quantize_weight_f8(empty(2, 2, 8, 16)), lambda op: op.quantize_weight_f8(empty(0, 16)),
    # a weight of one expert is no dense weight, nor the other way round
    lambda op: op.linear_f8(empty(3, 256, dtype=F8), empty(3, 2), empty(1, 40, 256, dtype=F8), empty(1, 1, 2), None,
                            torch.float16),
    lambda op: op.linear_f8(empty(3, 24, dtype=F8), empty(3, 1), empty(40, 24, dtype=F8), empty(1, 1), None,
                            torch.float16),
    lambda op: grouped(op, wq=empty(40, 256, dtype=F8), ws=empty(1, 2)),
    lambda op: grouped(op, xq=empty(2, 3, 256, dtype=F8), xs=empty(2, 3, 2)),
    lambda op: grouped(op, off=empty(4, dtype=torch.int32)), lambda op: grouped(op, off=empty(5, dtype=torch.int64)),
    lambda op: grouped(op, rows=empty(6, 1, dtype=torch.int32)), lambda op: grouped(op, rows=empty(6, dtype=torch.int64)),
])
def test_shape_functions_refuse_what_the_calls_refuse(call):
    """On meta tensors (as under a compiler) these gave shapes for calls that raise on the GPU."""
    with pytest.raises(ValueError):
        call(torch.ops.lowbit)


def grouped(op, **kw):
    a = dict(xq=empty(3, 256, dtype=F8), xs=empty(3, 2), rows=empty(6, dtype=torch.int32), off=empty(5, dtype=torch.int32),
             wq=empty(4, 40, 256, dtype=F8), ws=empty(4, 1, 2))
    a.update(kw)
    return op.linear_f8_grouped(a["xq"], a["xs"], a["rows"], a["off"], a["wq"], a["ws"], None, torch.bfloat16)


def test_shape_functions_take_what_the_calls_take():
    assert grouped(torch.ops.lowbit).shape == (6, 40) and grouped(torch.ops.lowbit, rows=None).shape == (3, 40)
    q, s = torch.ops.lowbit.quantize_weight_f8(empty(2, 130, 272, dtype=torch.float64))
    assert q.shape == (2, 130, 272) and s.shape == (2, 2, 3)
