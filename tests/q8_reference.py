"""The 8-bit form and its products in plain numpy, 64 bits: what the library's
results are compared with. Written from the definition in include/q8_linear.h;
shares no code with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3, E5M2 = 0, 1
# exponent of the largest value (1.75 * 2^emax), mantissa bits, smallest normal exponent, bias
FORMAT = {E4M3: (8, 3, -6, 7), E5M2: (15, 2, -14, 15)}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def ld(k: int) -> int:
    return -(-k // 16) * 16


def scale_index(r, k, K: int):
    g = -(-(-(-K // BLOCK)) // 4)
    return ((r // 128) * g + k // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + k % 4


def encode(y: np.ndarray, fmt: int) -> np.ndarray:
    """Bits of y rounded to nearest even (|y| at most the largest value; NaN allowed)."""
    _, mant, emin, bias = FORMAT[fmt]
    nan = np.isnan(y)
    a = np.abs(np.where(nan, 0.0, y))
    e = np.where(a > 0, np.maximum(np.frexp(a)[1] - 1, emin), emin)
    m = np.rint(np.ldexp(a, mant - e)).astype(np.int64)  # 0 .. 2^(mant+1)
    code = (e + bias - 1) * (1 << mant) + m  # subnormals: e = emin, m < 2^mant
    code = np.where(np.signbit(y), code | 0x80, code)
    return np.where(nan, 0x7F, code).astype(np.uint8)


def decode(bits: np.ndarray, fmt: int) -> np.ndarray:
    _, mant, emin, bias = FORMAT[fmt]
    b = bits.astype(np.int64)
    e, m = (b & 0x7F) >> mant, b & ((1 << mant) - 1)
    v = np.where(e == 0, np.ldexp(m.astype(float), emin - mant), np.ldexp((m + (1 << mant)).astype(float), e - bias - mant))
    if fmt == E4M3:
        v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where((b & 0x7F) > 0x7C, np.nan, np.where((b & 0x7F) == 0x7C, np.inf, v))
    return np.where(b & 0x80, -v, v)


def quantize(x: np.ndarray, fmt: int):
    """x (rows x K, float64) -> (values rows x ld, scale bytes, what they stand for)."""
    emax = FORMAT[fmt][0]
    rows, K = x.shape
    kb = -(-K // BLOCK)
    xb = np.zeros((rows, kb * BLOCK))
    xb[:, :K] = x
    xb = xb.reshape(rows, kb, BLOCK)
    fin = np.isfinite(xb)
    amax = np.where(fin, np.abs(xb), 0.0).max(2, initial=0.0)
    m, e = np.frexp(amax)
    s = np.where(amax > 0, np.maximum(e - 1 - emax + (m > 0.875), -127), 0)
    y = np.where(fin, np.ldexp(np.where(fin, xb, 0.0), -s[:, :, None]), np.nan)
    bits = encode(y, fmt)
    value = np.ldexp(decode(bits, fmt), s[:, :, None]).reshape(rows, kb * BLOCK)[:, :K]
    scales = np.full(-(-rows // 128) * 512 * -(-kb // 4), 127, dtype=np.uint8)
    if rows and kb:
        r, k = np.meshgrid(np.arange(rows), np.arange(kb), indexing="ij")
        scales[scale_index(r, k, K)] = s + 127
    out = np.zeros((rows, ld(K)), dtype=np.uint8)
    out[:, :K] = bits.reshape(rows, kb * BLOCK)[:, :K]
    return out, scales, value


def product_bound(a: np.ndarray, b: np.ndarray, dtype: str, extra=0.0):
    """(A . B^T, how far a result may be from it). The 8-bit products are exact.
    A sum formed 32 products at a time in at least 24 bits, any term of a step cut
    at the step's largest, is off by at most 33 * 2^-24 of the sum of magnitudes in each of
    the ceil(K / 32) steps; the last rounding by half a step of the result.
    `extra`: added to the sum before it is rounded (a bias, old contents)."""
    ref = a @ b.T + extra
    steps = -(-a.shape[1] // 32) + 4
    mag = np.abs(a) @ np.abs(b).T + np.abs(extra)
    tol = steps * 33 * 2.0 ** -24 * mag
    return ref, tol + HALF_STEP[dtype] * (np.abs(ref) + tol)
