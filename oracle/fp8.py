"""8-bit floating point products with a scale for each block of 128 (oracle; test infrastructure only).

OCP e4m3: sign, four exponent bits (bias 7), three fraction bits; largest 448, subnormals in steps of 2^-9, one
NaN a sign and no infinities. Values v of a group share a scale

    s = max(RN_f32(max |v| / 448), 2^-126),    code = RN_e4m3(RN_f32(v / s))   (ties to even)

and the group becomes NaN where it holds an infinity or a NaN. Groups: 128 values along a row or a column, or a block of
128 x 128. Scales of rows (of columns, for the transposed form) lie by blocks of the depth: ``[ceil(K / 128), rows]``.
Products are evaluated in fp64 from the codes and scales.
"""
from __future__ import annotations

import numpy as np

from .glu import silu

LARGEST = 448.0
LEAST = np.float32(2.0 ** -126)


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes, by the format's definition."""
    out = np.empty(256)
    for c in range(256):
        sign, exponent, fraction = -1.0 if c >> 7 else 1.0, (c >> 3) & 15, c & 7
        if exponent == 15 and fraction == 7:
            out[c] = np.nan
        elif exponent == 0:
            out[c] = sign * fraction * 2.0 ** -9
        else:
            out[c] = sign * (1 + fraction / 8) * 2.0 ** (exponent - 7)
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # 0 .. 448, rising


def to_e4m3(v: np.ndarray) -> np.ndarray:
    """The nearest code of values up to 448 (ties to the even code, as its last bit is the fraction's; NaN to NaN)."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isnan(v), 127, code) + 128 * np.signbit(v)
    return code.astype(np.uint8)


def from_e4m3(codes: np.ndarray) -> np.ndarray:
    return _VALUES[np.asarray(codes, dtype=np.uint8)]


def scale_of(group: np.ndarray) -> np.float32:
    group = np.asarray(group, dtype=np.float32)
    if not np.all(np.isfinite(group)):
        return np.float32(np.nan)
    most = np.max(np.abs(group)) if group.size else np.float32(0)
    return max(np.float32(most / np.float32(LARGEST)), LEAST)


def _codes_of(v, s):
    v = np.asarray(v, dtype=np.float32)
    if np.isnan(s):
        return np.full(v.shape, 127, dtype=np.uint8)
    return to_e4m3((v / np.float32(s)).astype(np.float32))


def quantize_rows(x: np.ndarray):
    """``(codes[M, K], scales[ceil(K/128), M])`` of fp32-exact values ``x[M, K]``."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    codes = np.zeros((M, K), dtype=np.uint8)
    scales = np.zeros((-(-K // 128), M), dtype=np.float32)
    for b in range(scales.shape[0]):
        k = slice(128 * b, 128 * b + 128)
        for m in range(M):
            scales[b, m] = scale_of(x[m, k])
            codes[m, k] = _codes_of(x[m, k], scales[b, m])
    return codes, scales


def quantize_columns(x: np.ndarray):
    """``(codes[K, M'], scales[ceil(M/128), K])``, M' the next multiple of 16, zero codes behind the last row."""
    codes, scales = quantize_rows(np.asarray(x, dtype=np.float32).T)
    pad = -codes.shape[1] % 16
    return np.concatenate([codes, np.zeros((codes.shape[0], pad), dtype=np.uint8)], axis=1), scales


def quantize_weight(w: np.ndarray):
    """``(codes[N, K], scales[ceil(N/128), ceil(K/128)])``: blocks of 128 x 128."""
    w = np.asarray(w, dtype=np.float32)
    N, K = w.shape
    codes = np.zeros((N, K), dtype=np.uint8)
    scales = np.zeros((-(-N // 128), -(-K // 128)), dtype=np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128)
            scales[i, j] = scale_of(w[at])
            codes[at] = _codes_of(w[at], scales[i, j])
    return codes, scales


def rows_value(codes, scales):
    """What codes ``[M, K]`` with scales ``[ceil(K/128), M]`` stand for."""
    return from_e4m3(codes) * np.repeat(np.asarray(scales, dtype=np.float64).T, 128, axis=1)[:, : codes.shape[1]]


def weight_value(codes, scales, halves: int = 1):
    """What a weight's codes ``[N, K]`` stand for; each of its ``halves`` has blocks of its own."""
    parts = zip(np.split(codes, halves), np.split(np.asarray(scales, dtype=np.float64), halves))
    return np.concatenate([from_e4m3(c) * np.repeat(np.repeat(s, 128, 0)[: c.shape[0]], 128, 1)[:, : c.shape[1]]
                           for c, s in parts])


def gemm_fp8_ref(x_value, w_value):
    return np.asarray(x_value, dtype=np.float64) @ np.asarray(w_value, dtype=np.float64).T


def swiglu_fp8_ref(x_value, w_value):
    y = gemm_fp8_ref(x_value, w_value)
    g, u = np.split(y, 2, axis=1)
    return silu(g) * u


def backward_fp8_ref(dy, x, wt_value):
    """``(dx, dw)`` of fp32-exact ``dy[M, N]``, ``x[M, K]`` and the value of the transposed weight ``[K, N]``."""
    dx = rows_value(*quantize_rows(dy)) @ np.asarray(wt_value).T
    dyc, dys = quantize_columns(dy)
    xc, xs = quantize_columns(x)
    return dx, rows_value(dyc, dys) @ rows_value(xc, xs).T
