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


def reference(t):
    with np.errstate(all="ignore"):
        return o.lora(f64(t["x"]), f64(t["a"]), f64(t["b"]), f64(t["scales"]), t["ids"].numpy(), f64(t["base"]))


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
