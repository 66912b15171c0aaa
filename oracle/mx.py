"""Microscaled (MX) formats, the RMS norm that ends in them and products of them,
in fp64 numpy from the formats' definitions. Test infrastructure; shares no
code with the library.

A block of 32 consecutive elements of a row shares 2^e. Element values are
enumerated (E2M1: 8 magnitudes, E4M3: 127) and a value is rounded by searching
the list, ties to the code whose last bit is 0.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
E4M3, E2M1 = 0, 1


def _magnitudes(exp_bits: int, man_bits: int, count: int) -> np.ndarray:
    """Values of codes 0 .. count - 1 of a float with the usual bias and subnormals."""
    bias = 2 ** (exp_bits - 1) - 1
    out = []
    for code in range(count):
        e, m = code >> man_bits, code & ((1 << man_bits) - 1)
        out.append(np.ldexp(m / 2.0 ** man_bits, 1 - bias) if e == 0 else np.ldexp(1.0 + m / 2.0 ** man_bits, e - bias))
    return np.array(out, dtype=np.float64)


# E4M3's code 127 is NaN (and it has no infinities); E2M1 has neither.
MAGNITUDES = {E2M1: _magnitudes(2, 1, 8), E4M3: _magnitudes(4, 3, 127)}
EMAX = {E2M1: 2, E4M3: 8}
SIGN = {E2M1: 8, E4M3: 128}


def encode(v: np.ndarray, fmt: int) -> np.ndarray:
    """Codes of fp64 values: nearest, ties to even codes, saturated."""
    table = MAGNITUDES[fmt]
    a = np.abs(v)
    hi = np.searchsorted(table, a).clip(0, len(table) - 1)
    lo = (hi - 1).clip(0)
    d_hi, d_lo = table[hi] - a, a - table[lo]
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= table[-1], len(table) - 1, code)
    return (code + np.where(np.signbit(v), SIGN[fmt], 0)).astype(np.uint8)


def decode(code: np.ndarray, fmt: int) -> np.ndarray:
    mag = np.append(MAGNITUDES[fmt], np.nan) if fmt == E4M3 else MAGNITUDES[fmt]
    sign = (code.astype(np.int64) & SIGN[fmt]) != 0
    v = mag[code.astype(np.int64) & (SIGN[fmt] - 1)]
    return np.where(sign, -v, v)


def quantize(x: np.ndarray, fmt: int):
    """fp64 [rows, cols] -> (codes [rows, cols], scale bytes [rows, cols / 32])."""
    rows, cols = x.shape
    b = np.asarray(x, dtype=np.float64).reshape(rows, cols // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=-1)
    amax = np.where(bad, 1.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=-1))
    _, ex = np.frexp(amax)
    e = np.where(amax > 0, np.maximum(ex - 1 - EMAX[fmt], -127), -127)
    codes = encode(np.ldexp(np.where(bad[..., None], 0.0, b), -e[..., None]), fmt)
    codes = np.where(bad[..., None], 0, codes).reshape(rows, cols).astype(np.uint8)
    return codes, np.where(bad, 255, e + 127).astype(np.uint8)


def dequantize(codes: np.ndarray, scales: np.ndarray, fmt: int) -> np.ndarray:
    """fp64 values of codes [rows, cols] with scale bytes [rows, cols / 32]."""
    rows, cols = codes.shape
    v = decode(codes, fmt).reshape(rows, cols // BLOCK, BLOCK)
    out = np.ldexp(v, scales.astype(np.int64)[..., None] - 127)
    return np.where((scales == 255)[..., None], np.nan, out).reshape(rows, cols)


def pack(codes: np.ndarray, scales: np.ndarray, fmt: int):
    """The library's storage: (data [rows, kp or kp / 2], scales [kp / 128, rows, 4])."""
    rows, cols = codes.shape
    kp = (cols + 127) // 128 * 128
    data = np.zeros((rows, kp), np.uint8)
    data[:, :cols] = codes
    if fmt == E2M1:
        data = data[:, 0::2] | (data[:, 1::2] << 4)
    sc = np.full((rows, kp // BLOCK), 127, np.uint8)
    sc[:, :cols // BLOCK] = scales
    return np.ascontiguousarray(data), np.ascontiguousarray(sc.reshape(rows, kp // 128, 4).transpose(1, 0, 2))


def unpack(data: np.ndarray, scales: np.ndarray, rows: int, cols: int, fmt: int):
    """Inverse of pack, padding dropped."""
    kp = (cols + 127) // 128 * 128
    if fmt == E2M1:
        d = data.reshape(rows, kp // 2)
        codes = np.stack((d & 15, d >> 4), -1).reshape(rows, kp)
    else:
        codes = data.reshape(rows, kp)
    sc = scales.reshape(kp // 128, rows, 4).transpose(1, 0, 2).reshape(rows, kp // BLOCK)
    return codes[:, :cols], sc[:, :cols // BLOCK]


def rmsnorm(h: np.ndarray, gamma: np.ndarray, eps: float) -> np.ndarray:
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        return h / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps) * gamma


def grouped(x: np.ndarray, w: np.ndarray, offsets) -> np.ndarray:
    """x [M, K] against w [E, N, K]: rows offsets[e] .. offsets[e + 1] with expert e; others NaN."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            y[a:b] = x[a:b] @ w[e].T
    return y
