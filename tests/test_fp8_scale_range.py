"""8-bit products whose two scales multiply to more than fp32 holds, or to less, on every kernel that the sizes
pick: what fp4q.h says of them.

A block's sum is exact here (one value of A and one of B throughout the block; 0, or 2^-18 to 2^25 in
magnitude), and the other blocks are zeros.  u = 2^-24.
 - 2^-126 <= |sa sb| < 2^128: the multiplier is rounded once (u), the multiply-add once (u, or half a step
   of fp32's subnormal numbers): 2 u |ref| + 2^-150.
 - below, the multiplier is rounded to fp32's subnormal numbers, by 2^-150 at most, or to 0: |sum| 2^-150 more.
 - where the tensor core applies the scales (E8M0), each of the 33 terms of a block's four MMAs may
   lose a step of 2^-149 instead: 132 of them.
 - above: the formula's value, infinity of the sum's sign, or NaN where the sum is 0."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as o

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32_MAX = float(np.finfo(np.float32).max)

VALUES = np.array([0.0, 2.0 ** -9, 1.0, -448.0])
A_SCALES = {o.F32: np.array([1.0, 2.0 ** 100, 2.0 ** 127, 1.3 * 2.0 ** -70, 1.5 * 2.0 ** -126, 2.0 ** -149, 0.0,
                             1.7 * 2.0 ** 64, -(2.0 ** 100), F32_MAX, 1.1 * 2.0 ** -40], np.float32),
            o.E8M0: np.array([127, 227, 254, 57, 0, 1, 190, 100, 30], np.uint8)}
B_SCALES = {o.F32: np.array([1.0, 2.0 ** 30, 2.0 ** 127, 1.7 * 2.0 ** -70, 1.7 * 2.0 ** -20, 2.0 ** -126, 1.9 * 2.0 ** 63,
                             0.0, -1.9 * 2.0 ** -100], np.float32),
            o.E8M0: np.array([127, 157, 254, 57, 107, 0, 1, 191, 60], np.uint8)}

# few rows (one CTA, and K over several), 128 x 128, 256 x 128 and the widest tiles
SHAPES = [(16, 1160, 272), (9, 1160, 1040), (32, 1160, 272), (64, 1160, 272), (60, 1160, 1040), (514, 2050, 272),
          (1180, 1160, 1040), (1032, 2056, 272), (2500, 2056, 272)]


@pytest.fixture(scope="module")
def F(cuda_device):
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


def codes(values, K, block):
    """[len(values)][K] of zeros but for the block, which holds a row's value."""
    c = np.zeros((len(values), K), np.uint8)
    c[:, 128 * block:128 * block + 128] = o.e4m3_encode(values)[:, None]
    return torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)


def scales(values, kb, block, fmt):
    s = np.full((len(values), kb), 1.0 if fmt == o.F32 else 127, values.dtype)
    s[:, block] = values
    t = torch.from_numpy(s).cuda()
    return t if fmt == o.F32 else t.view(torch.float8_e8m0fnu)


@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_of_scales_past_fp32(F, M, N, K, fmt):
    kb, block = -(-K // 128), 1
    m, n, t = np.arange(M), np.arange(N), np.arange(-(-N // 128))
    pool_a, pool_b = A_SCALES[fmt], B_SCALES[fmt]
    for turn in range(2):   # both with all scales against all, values against values
        va, vb = VALUES[(m // len(pool_a) + turn) % 4], VALUES[(n + turn) % 4]
        sa, sb = pool_a[(m + 5 * turn) % len(pool_a)], pool_b[(t + 4 * turn) % len(pool_b)]
        d = F.gemm_fp8(codes(va, K, block), scales(sa, kb, block, fmt), codes(vb, K, block),
                       scales(sb, kb, block, fmt), out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert F.fp4q_device_status() == F.FP4Q_OK
        got = d.cpu().numpy().astype(np.float64)
        sums = 128.0 * np.outer(va, vb)
        mult = np.outer(o.scale_values(sa), np.repeat(o.scale_values(sb), 128)[:N])
        ref = sums * mult
        past = np.abs(mult) >= 2.0 ** 128
        tol = 2 * U * np.abs(ref) + 2.0 ** -150 * (1 + np.abs(sums) * (np.abs(mult) < 2.0 ** -126))
        if fmt == o.E8M0:
            tol += 132 * 2.0 ** -149
        # within the range: the formula, infinite where fp32 is passed
        over = ~past & (np.abs(ref) * (1 - 2 * U) >= 2.0 ** 128)
        inside = ~past & (np.abs(ref) * (1 + 2 * U) <= F32_MAX)
        assert np.all(np.isinf(got[over])) and np.all(np.sign(got[over]) == np.sign(ref[over]))
        err = np.abs(got - ref)
        assert np.all(err[inside] <= tol[inside]), float(np.max(err[inside] / tol[inside]))
        # past it
        infinite = (got == np.inf) & (ref > 0) | (got == -np.inf) & (ref < 0)
        stated = np.where(sums == 0, np.isnan(got) | (got == 0), infinite | (err <= 2 * U * np.abs(ref)))
        assert np.all(stated[past])
        assert np.count_nonzero(past) > 0.05 * past.size and np.count_nonzero(inside) > 0.3 * past.size


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_scales_that_are_no_numbers(F, M, N, K):
    """An infinite or NaN fp32 scale follows the formula: infinity times the block's sum, and NaN where that
    sum is zero."""
    kb, block = -(-K // 128), 1
    rng = np.random.default_rng(1)
    va, vb = VALUES[rng.integers(0, 4, M)], VALUES[rng.integers(0, 4, N)]
    sa = np.array([1.0, np.inf, -np.inf, np.nan, 1.5], np.float32)[np.arange(M) % 5]
    sb = np.array([1.0, 2.0 ** 100, -1.0, np.inf, 2.0 ** -100], np.float32)[np.arange(-(-N // 128)) % 5]
    d = F.gemm_fp8(codes(va, K, block), scales(sa, kb, block, o.F32), codes(vb, K, block), scales(sb, kb, block, o.F32),
                   out_dtype=torch.float32)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        ref = 128.0 * np.outer(va, vb) * np.outer(sa.astype(np.float64), np.repeat(sb.astype(np.float64), 128)[:N])
    got = d.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(np.isinf(got), np.isinf(ref)) and np.array_equal(np.sign(got[np.isinf(got)]), np.sign(ref[np.isinf(ref)]))
    ok = np.isfinite(ref)
    assert np.all(np.abs(got[ok] - ref[ok]) <= 2 * U * np.abs(ref[ok]))
