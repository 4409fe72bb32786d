"""Which kernel the 8-bit GEMM takes."""

import random

import pytest

from oracle import fp8_oracle as o

SMS = 148
FORMATS = [o.F32, o.E8M0]


@pytest.fixture(scope="module")
def lib():
    from microscaling_fp4_quantization_b200 import build
    build.build()
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


# tiles of many rows: (M, N, K) with columns added to N for rows of no alignment
MANY = {(o.F32, (128, 128)): (1880, 520, 400), (o.F32, (256, 128)): (1055, 4104, 144), (o.F32, (256, 256)): (527, 4104, 272),
        (o.E8M0, (128, 128)): (1880, 520, 400), (o.E8M0, (256, 224)): (527, 4104, 272)}


def test_no_other_kernel_is_chosen(lib):
    """Over sizes and SM counts: no tile but those that the tests run."""
    seen = set()
    rng = random.Random(0)
    for _ in range(50000):
        M, N, K = (int(2 ** rng.uniform(0, 17)) for _ in range(3))
        fmt, sms = rng.randint(0, 1), rng.choice([SMS, SMS, 132, 75, 20, 2])
        tm, tn, split = lib.fp4q_selftest_gemm_fp8_choice(fmt, M, N, 16 * -(-K // 64), sms)
        assert 1 <= split <= 8 and (tm <= 64 or split == 1)
        seen.add((fmt, (tm, tn)))
    assert seen == set(MANY) | {(fmt, (rows, 128)) for fmt in FORMATS for rows in (16, 32, 64)}


def test_refusals(lib):
    import ctypes
    v = [ctypes.byref(ctypes.c_int()) for _ in range(3)]
    def q(fmt=0, M=4, N=4, K=128, sms=SMS, out=v):
        return lib.raw_call("fp4q_selftest_gemm_fp8_choice", fmt, M, N, K, sms, *out)
    assert q() == lib.FP4Q_OK
    assert q(fmt=2) == lib.FP4Q_ERR_UNSUPPORTED
    for bad in (dict(sms=-1), dict(sms=1), dict(out=[None] + v[1:]), dict(out=v[:2] + [None])):
        assert q(**bad) == lib.FP4Q_ERR_ARG, bad
    for bad in (dict(M=0), dict(N=0), dict(K=0), dict(K=24), dict(M=-1), dict(M=1 << 31), dict(M=1 << 30, N=1 << 30)):
        assert q(**bad) == lib.FP4Q_ERR_SHAPE, bad
