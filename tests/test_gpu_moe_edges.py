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
