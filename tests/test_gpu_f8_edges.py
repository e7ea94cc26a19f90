"""The 8-bit path on the GPU at the ends of its ranges: huge rows, large grids, wide scales, the
accuracy of 16-bit outputs, and cast or shared modules."""
import numpy as np
import pytest
import torch

from bit_groupwise_weight_amd import lowbit as lb
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
