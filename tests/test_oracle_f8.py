"""Pins of the 8-bit path's oracle: the e4m3 table against the format's constants, rounding against
a brute-force search, span scales at their borders, and the products against a scalar loop."""
import numpy as np
import pytest

from oracle import f8_oracle as o


def test_table_constants():
    assert o.E4M3[0x7e] == 448.0 and o.E4M3[0x01] == 2.0 ** -9 and o.E4M3[0x08] == 2.0 ** -6
    assert o.E4M3[0x38] == 1.0 and o.E4M3[0xb8] == -1.0 and o.E4M3[0x39] == 1.125
    assert np.isnan(o.E4M3[0x7f]) and np.isnan(o.E4M3[0xff])
    assert np.all(np.diff(o.E4M3[:127]) > 0)


def test_rounding_is_nearest_ties_to_even():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-460, 460, 2000), rng.uniform(-0.02, 0.02, 2000),
                        o.E4M3[:127], -o.E4M3[:127], (o.E4M3[:126] + o.E4M3[1:127]) / 2, [0.0, 464.0]])
    got = o.e4m3_round(v)
    pats = np.array([p for p in range(256) if not np.isnan(o.E4M3[p])])
    for x, g in zip(v, got):
        d = np.abs(o.E4M3[pats] - x)
        near = pats[d == d.min()]
        assert g in near
        if np.abs(o.E4M3[near]).max() != np.abs(o.E4M3[near]).min():      # a tie
            assert g % 2 == 0


def test_rounding_agrees_with_torch():
    import torch
    v = np.random.default_rng(1).uniform(-448, 448, 4096).astype(np.float32)
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o.e4m3_round(v), t)


@pytest.mark.parametrize("amax, scale", [(0.0, 0.0), (2.0 ** -111, 0.0), (2.0 ** -110, None),
                                         (3.4e38, None), (np.inf, np.nan), (np.nan, np.nan)])
def test_span_scale_borders(amax, scale):
    v = np.zeros(128, np.float32)
    v[5] = amax
    s, f = o.span_scale(v, 448.0)
    if scale is None:
        assert s == np.float32(amax) / np.float32(448) and s > 0 and np.isfinite(f)
    elif np.isnan(scale):
        assert np.isnan(s)
    else:
        assert s == 0 and f == 0


def test_quantized_values_are_within_half_a_step():
    x = np.random.default_rng(2).standard_normal((7, 272)).astype(np.float32)
    q, s = o.quantize_f8_rows(x)
    assert s.shape == (7, 3)
    full = np.repeat(s, 128, 1)[:, :272].astype(np.float64)
    err = np.abs(o.E4M3[q] * full - x)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * full) * (1 + 2.0 ** -20))


def test_linear_against_a_scalar_loop():
    rng = np.random.default_rng(3)
    M, N, K = 3, 131, 144
    xq, wq = rng.integers(0, 127, (M, K)).astype(np.uint8), rng.integers(0, 127, (N, K)).astype(np.uint8)
    xs, ws = rng.random((M, 2)).astype(np.float32), rng.random((2, 2)).astype(np.float32)
    y, A = o.linear_f8(xq, xs, wq, ws)
    for m, n in [(0, 0), (2, 130), (1, 127), (1, 128)]:
        want = sum(float(xs[m, k // 128]) * float(ws[n // 128, k // 128]) * o.E4M3[xq[m, k]] * o.E4M3[wq[n, k]]
                   for k in range(K))
        assert abs(y[m, n] - want) <= 1e-12 * A[m, n]
    off = np.array([0, 2, 2, 3])
    w3, s3 = np.stack([wq, wq, wq]), np.stack([ws, ws, 2 * ws])
    rows = np.array([1, 1, 2, 0])
    yg, _ = o.linear_f8_grouped(xq, xs, rows, off, w3, s3, None, np.full((4, N), 7.0))
    assert np.array_equal(yg[0], y[1]) and np.array_equal(yg[1], y[1])
    assert np.allclose(yg[2], 2 * y[2], rtol=1e-14) and np.all(yg[3] == 7.0)
