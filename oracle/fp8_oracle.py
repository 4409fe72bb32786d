"""Plain CPU restatement of the 8-bit linear-layer operators (TEST INFRASTRUCTURE): E4M3 codes with
a scale per 128 channels, the RMS norm that ends in them, and the product of two such operands.
It follows the rules written in ``include/fp4q.h`` (fp4q_quantize_fp8, fp4q_add_rmsnorm_fp8,
fp4q_gemm_fp8), in numpy, with a search over the E4M3 values in place of a conversion."""

from __future__ import annotations

import numpy as np

F32, E8M0 = 0, 1
BLOCK = 128

_C = np.arange(127)
MAGNITUDES = np.where(_C >> 3 == 0, (_C & 7) * 2.0 ** -9, (1 + (_C & 7) / 8) * np.ldexp(1.0, (_C >> 3) - 7))
_MIDPOINTS = (MAGNITUDES[:-1] + MAGNITUDES[1:]) / 2


def e4m3_encode(v) -> np.ndarray:
    """float64 -> E4M3 byte: nearest, ties to the even code, saturating at 448, NaN -> 0x7F."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    i = np.searchsorted(_MIDPOINTS, a, side="left")           # the lower code on a midpoint
    tie = (i < 126) & (a == _MIDPOINTS[np.minimum(i, 125)])
    i = i + (tie & (i % 2 == 1))
    c = np.minimum(i, 126) | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isnan(v), 0x7F, c).astype(np.uint8)


def e4m3_decode(codes) -> np.ndarray:
    c = np.asarray(codes, np.uint8)
    m = np.append(MAGNITUDES, np.nan)[c & 0x7F]
    return np.where(c & 0x80, -m, m)


def e8m0_decode(b) -> np.ndarray:
    b = np.asarray(b, np.int64)
    return np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))


def scale_of(A, fmt):
    """Largest magnitudes A -> (stored scales: float32, or E8M0 bytes; their values in float64)."""
    A = np.asarray(A, np.float64)
    ok = np.isfinite(A)
    Af = np.where(ok, A, 1.0)
    if fmt == F32:
        s = np.maximum(Af.astype(np.float32) / np.float32(448), np.float32(2.0 ** -126))
        s = np.where(ok, s, np.float32(np.nan)).astype(np.float32)
        return s, s.astype(np.float64)
    byte = np.full(A.shape, 1, np.int64)                      # the least e with 448 2^e >= A, by trial
    for b in range(2, 255):
        byte = np.where(448.0 * np.ldexp(1.0, b - 1 - 127) < Af, b, byte)
    byte = np.where(ok, byte, 255)
    return byte.astype(np.uint8), e8m0_decode(byte)


def blocks_amax(y, rows):
    """[M][K] -> largest magnitude of each block of rows x 128 (NaN where it holds one)."""
    M, K = y.shape
    out = np.empty((-(-M // rows), -(-K // BLOCK)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.max(np.abs(y[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK]))
    return out


def spread(s, rows, M, K):
    """Block values [.., ..] -> one per element [M][K]."""
    return np.repeat(np.repeat(s, rows, 0)[:M], BLOCK, 1)[:, :K]


def quantize(x, rows, fmt):
    """x: float32 [M][K] -> (codes, stored scales)."""
    x = np.asarray(x, np.float32)
    stored, s = scale_of(blocks_amax(x.astype(np.float64), rows), fmt)
    with np.errstate(all="ignore"):
        q = x / spread(s, rows, *x.shape).astype(np.float32)   # fp32, correctly rounded
    return e4m3_encode(q.astype(np.float64)), stored


def rmsnorm(x, residual, weight, eps):
    """(h, y) in float64."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    with np.errstate(all="ignore"):
        return h, h / np.sqrt(np.mean(h * h, 1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def scale_values(stored):
    return e8m0_decode(stored) if stored.dtype == np.uint8 else stored.astype(np.float64)


def operand(codes, stored, rows):
    return e4m3_decode(codes) * spread(scale_values(stored), rows, *codes.shape)


def gemm(a_codes, a_scales, b_codes, b_scales):
    return operand(a_codes, a_scales, 1) @ operand(b_codes, b_scales, BLOCK).T
