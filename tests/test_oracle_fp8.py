"""Pins of the 8-bit oracle (CPU): hand-worked codes, scales and products, and torch's own E4M3
conversion as a second route."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as o


def test_hand_worked_codes():
    """1.0 = 0x38; 448 = 0x7E; 2^-9 = 0x01; 17 lies between 16 (0x58) and 18 (0x59): tie to the even
    code; 19 between 18 (0x59) and 20 (0x5A): tie to 0x5A; 2^-10 between 0 and 2^-9: tie to 0."""
    v = [0.0, -0.0, 1.0, -1.0, 448.0, 1e6, 2.0 ** -9, 17.0, 19.0, 2.0 ** -10, -(2.0 ** -10) * 1.001, np.nan]
    c = [0x00, 0x80, 0x38, 0xB8, 0x7E, 0x7E, 0x01, 0x58, 0x5A, 0x00, 0x81, 0x7F]
    assert o.e4m3_encode(v).tolist() == c


def test_codes_agree_with_torch():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.integers(-4, 3, 20000), o.MAGNITUDES, -o.MAGNITUDES,
                        o._MIDPOINTS]).astype(np.float32)
    t = torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o.e4m3_encode(v), t)
    every = np.arange(256, dtype=np.uint8)
    d = torch.from_numpy(every).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(o.e4m3_decode(every), d, equal_nan=True)


def test_hand_worked_scales():
    A = np.array([448.0, 449.0, 896.0, 0.0, 1.0, np.inf, np.nan, 224.0])
    s, v = o.scale_of(A, o.F32)
    assert s[0] == 1 and s[2] == 2 and s[3] == np.float32(2.0 ** -126) and s[4] == np.float32(1 / 448) and s[7] == 0.5
    assert np.isnan(s[5:7]).all()
    b, v = o.scale_of(A, o.E8M0)
    # 1 / 448 = 2^-8.8: 2^-8
    assert b.tolist() == [127, 128, 128, 1, 119, 255, 255, 126] and v[1] == 2.0


def test_hand_worked_product():
    """Two K-blocks of A (scales 2, 0.5) against two of B (scales 1, 4): 128 * 1*1 * 2 * 1 + 16 * 2*3 *
    0.5 * 4 = 448."""
    a = o.e4m3_encode(np.array([[1.0] * 128 + [2.0] * 16]))
    b = o.e4m3_encode(np.array([[1.0] * 128 + [3.0] * 16]))
    for f in (lambda v: np.asarray(v, np.float32), lambda v: (np.log2(v) + 127).astype(np.uint8)):
        assert o.gemm(a, f([[2.0, 0.5]]), b, f([[1.0, 4.0]])).tolist() == [[448.0]]


@pytest.mark.parametrize("fmt", [o.F32, o.E8M0])
@pytest.mark.parametrize("rows", [1, 128])
def test_quantized_values_are_near(fmt, rows):
    """A code is off by at most half a step (2^-4 of the value, or 2^-10 of the scale for the smallest);
    with E8M0 the block maximum lies in (224, 448] scales."""
    x = (np.random.default_rng(1).standard_normal((130, 272)) * 3).astype(np.float32)
    c, s = o.quantize(x, rows, fmt)
    sv = o.spread(o.scale_values(s), rows, *x.shape)
    err = np.abs(o.operand(c, s, rows) - x)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * sv) * (1 + 1e-6))
    top = o.blocks_amax(np.abs(x / sv), rows)
    assert np.all(top <= 448 * (1 + 1e-6)) and np.all(top > 223.9)


def test_norm_of_ones():
    h, y = o.rmsnorm(np.ones((1, 16)), np.ones((1, 16)), np.full(16, 3.0), 0.0)
    assert np.all(h == 2) and np.allclose(y, 3)
