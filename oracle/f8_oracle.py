"""CPU oracle of the 8-bit path (test infrastructure only, plain numpy): e4m3 codes with a scale
for each block of 128, the residual-add RMS norm, and the block-scaled product, dense and grouped.

  e4m3      the OCP numbers of 1 sign, 4 exponent (bias 7) and 3 mantissa bits: no infinities,
            one NaN pattern per sign, largest 448, smallest 2^-9.  Rounding is a search in the
            table of all of them: nearest, ties to the even pattern.
  quantize  per span: s = fp32(max |v| / top), code = round(fp32(v * fp32(top / max |v|))), with
            top = 448 (e4m3) or 127 (int8); a span whose max |v| is below 2^-110 has scale 0 and
            codes 0, a span holding a NaN or an infinity has scale NaN and codes 0.
  norm      h = round(x + residual), y = h / sqrt(mean(h^2) + eps) * weight in float64.
  linear    sum_b xs[m, b] ws[n / 128, b] sum_{k in b} xq[m, k] wq[n, k] in float64, and the sum A
            of the products' magnitudes.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

BLOCK = 128


def _e4m3_values() -> np.ndarray:
    """Value of each of the 256 patterns, from the format's definition."""
    v = np.empty(256)
    for p in range(256):
        sign = -1.0 if p & 0x80 else 1.0
        e, m = (p >> 3) & 15, p & 7
        if e == 15 and m == 7:
            v[p] = np.nan
        elif e == 0:
            v[p] = sign * m * 2.0 ** -9
        else:
            v[p] = sign * (1.0 + m / 8.0) * 2.0 ** (e - 7)
    return v


E4M3 = _e4m3_values()
_POS = E4M3[:127]                     # 0 .. 448, ascending, pattern = index


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Patterns (uint8) of the nearest e4m3 numbers to float values of magnitude <= 464."""
    a = np.abs(v.astype(np.float64))
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (a >= _POS[hi])
    code = np.where(up, hi, lo).astype(np.uint8)
    return code | np.where(np.signbit(v), 0x80, 0).astype(np.uint8)


def span_scale(v: np.ndarray, top: float) -> Tuple[np.ndarray, np.ndarray]:
    """Scale and factor (fp32) of spans v[..., n] of fp32 values."""
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(-1)
        good = np.isfinite(v).all(-1)
        big = good & (amax >= np.float32(2.0 ** -110))
        safe = np.where(big, amax, np.float32(1)).astype(np.float32)
        s = np.where(big, safe / np.float32(top), np.float32(0)).astype(np.float32)
        f = np.where(big, np.float32(top) / safe, np.float32(0)).astype(np.float32)
    return np.where(good, s, np.float32(np.nan)).astype(np.float32), f


def _scaled(v: np.ndarray, f: np.ndarray) -> np.ndarray:
    return (np.where(np.isfinite(v), v, np.float32(0)) * f).astype(np.float32)


def quantize_f8_rows(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """x[M, K] fp32 -> patterns uint8 [M, K], scales fp32 [M, ceil(K / 128)]."""
    M, K = x.shape
    kb = -(-K // BLOCK)
    q, s = np.zeros((M, K), np.uint8), np.zeros((M, kb), np.float32)
    for b in range(kb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        s[:, b], f = span_scale(v, 448.0)
        codes = e4m3_round(_scaled(v, f[:, None]))
        q[:, b * BLOCK:(b + 1) * BLOCK] = np.where(np.isnan(s[:, b:b + 1]), 0, codes)
    return q, s


def quantize_f8_weight(w: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """w[N, K] fp32 -> patterns uint8 [N, K], scales fp32 [ceil(N / 128), ceil(K / 128)]."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    q, s = np.zeros((N, K), np.uint8), np.zeros((nb, kb), np.float32)
    for i in range(nb):
        for b in range(kb):
            at = np.s_[i * BLOCK:(i + 1) * BLOCK, b * BLOCK:(b + 1) * BLOCK]
            v = w[at]
            s[i, b], f = span_scale(v.reshape(-1), 448.0)
            q[at] = 0 if np.isnan(s[i, b]) else e4m3_round(_scaled(v, f))
    return q, s


def rmsnorm(h: np.ndarray, weight: Optional[np.ndarray], eps: float) -> np.ndarray:
    """y in float64 of rows h (already the rounded sum); rows with a NaN or infinity are NaN."""
    h = h.astype(np.float64)
    with np.errstate(all="ignore"):
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
        if weight is not None:
            y = y * weight.astype(np.float64)
    y[~np.isfinite(h).all(1)] = np.nan
    return y


def linear_f8(xq: np.ndarray, xs: np.ndarray, wq: np.ndarray, ws: np.ndarray,
              bias: Optional[np.ndarray] = None,
              columns: Optional[np.ndarray] = None) -> Tuple[np.ndarray, np.ndarray]:
    """(y, A) in float64 from patterns and scales; A sums the magnitudes of the products.
    `columns`: the weight rows to compute (all by default)."""
    columns = np.arange(wq.shape[0]) if columns is None else columns
    y, A = np.zeros((xq.shape[0], len(columns))), np.zeros((xq.shape[0], len(columns)))
    x, w = E4M3[xq], E4M3[wq[columns]]
    with np.errstate(all="ignore"):
        for b in range(xs.shape[1]):
            at = np.s_[:, b * BLOCK:(b + 1) * BLOCK]
            s = xs[:, b:b + 1].astype(np.float64) * ws[columns // BLOCK, b].astype(np.float64)[None, :]
            y += s * (x[at] @ w[at].T)
            A += np.abs(s) * (np.abs(x[at]) @ np.abs(w[at]).T)
    if bias is not None:
        b = bias[columns].astype(np.float64)
        y, A = y + b, A + np.abs(b)
    return y, A


def linear_f8_grouped(xq, xs, rows, offsets, wq, ws, bias, y0,
                      columns: Optional[np.ndarray] = None) -> Tuple[np.ndarray, np.ndarray]:
    """(y, A): y0 with the rows of every expert replaced; rows == None reads row t for row t."""
    columns = np.arange(wq.shape[1]) if columns is None else columns
    y = y0[:, columns].astype(np.float64)
    A = np.zeros(y.shape)
    source = np.arange(y.shape[0]) if rows is None else rows
    for e in range(wq.shape[0]):
        t = np.arange(offsets[e], offsets[e + 1])
        out = (source[t] < 0) | (source[t] >= xq.shape[0])
        y[t[out]] = np.nan
        t = t[~out]
        if len(t):
            r = source[t]
            y[t], A[t] = linear_f8(xq[r], xs[r], wq[e], ws[e], None if bias is None else bias[e], columns)
    return y, A
