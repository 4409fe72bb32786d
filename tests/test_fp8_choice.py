"""Every kernel of the 8-bit GEMM, with every scale format, output type, alignment of D's rows and split of K, at
sizes that pick it: the choice itself is asserted (on the CPU for 148 SMs, on the GPU for its own count).
Tolerances as in test_fp8.py."""

import random

import pytest
import torch

from oracle import fp8_oracle as o

SMS = 148
FORMATS = [o.F32, o.E8M0]
IDS = ["f32", "e8m0"]


@pytest.fixture(scope="module")
def lib():
    from microscaling_fp4_quantization_b200 import build
    build.build()
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


@pytest.fixture(scope="module")
def F(cuda_device):
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


def few_shape(rows, split, N):
    """M, N, K whose product takes tiles of `rows` tokens and, two blocks to a CTA, that split."""
    return {16: 13, 32: 27, 64: 50}[rows], N, 256 * split + (16 if split > 1 else 0)


# tiles of many rows: (M, N, K) with columns added to N for rows of no alignment
MANY = {(o.F32, (128, 128)): (1880, 520, 400), (o.F32, (256, 128)): (1055, 4104, 144), (o.F32, (256, 256)): (527, 4104, 272),
        (o.E8M0, (128, 128)): (1880, 520, 400), (o.E8M0, (256, 224)): (527, 4104, 272)}
# D's rows on whole 32 bytes (of 16-bit types), on 16, on 2 or 4 columns, and odd
ALIGNED, UNALIGNED = [0, 8], [2, 1]
FEW_N = [256, 136, 134, 133]
# tiles whose clusters may not all be resident: N / 128 of them, split as far as there are SMs
NATURAL = {18: 8, 19: 7, 21: 7, 24: 6, 29: 5, 36: 4, 37: 4, 49: 3, 74: 2, 75: 1}


def test_shapes_reach_what_they_name(lib):
    q = lib.fp4q_selftest_gemm_fp8_choice
    for fmt in FORMATS:
        for rows in (16, 32, 64):
            for split in range(1, 9):
                for N in FEW_N:
                    assert q(fmt, *few_shape(rows, split, N), SMS) == (rows, 128, split)
            for tiles, split in NATURAL.items():
                assert q(fmt, {16: 13, 32: 27, 64: 50}[rows], 128 * tiles - 100, 2064, SMS) == (rows, 128, split)
    for (fmt, tile), (M, N, K) in MANY.items():
        for more in ALIGNED + UNALIGNED:
            assert q(fmt, M, N + more, K, SMS) == tile + (1,)


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


def check(F, M, N, K, fmt, dtypes):
    from test_fp8 import check_gemm, make_operands, synced
    a, b = make_operands(F, M, N, K, fmt, M + N + K)
    size = max(t.itemsize for t in dtypes)
    raw = torch.empty(M * N * size + 64, dtype=torch.uint8, device="cuda")
    for dtype in dtypes:
        raw.fill_(0xA5)
        end = M * N * dtype.itemsize
        d = F.gemm_fp8(*a, *b, out=raw[:end].view(dtype).view(M, N))
        again = F.gemm_fp8(*a, *b, out_dtype=dtype)
        synced(F)
        check_gemm(d, a, b, K)
        assert torch.equal(d, again)
        assert torch.all(raw[end:] == 0xA5)


TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.gpu
@pytest.mark.parametrize("split", range(1, 9))
@pytest.mark.parametrize("rows", [16, 32, 64])
@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
def test_few_rows(F, fmt, rows, split):
    for N in FEW_N:
        M, N, K = few_shape(rows, split, N)
        assert F.fp4q_selftest_gemm_fp8_choice(fmt, M, N, K) == (rows, 128, split)
        check(F, M, N, K, fmt, TYPES)


@pytest.mark.gpu
@pytest.mark.parametrize("tiles", NATURAL)
@pytest.mark.parametrize("rows", [16, 32, 64])
def test_few_rows_as_split_as_there_are_sms(F, rows, tiles):
    check(F, {16: 13, 32: 27, 64: 50}[rows], 128 * tiles - 100, 2064, o.F32, TYPES[:1])


@pytest.mark.gpu
@pytest.mark.parametrize("more", ALIGNED + UNALIGNED)
@pytest.mark.parametrize("which", MANY, ids=lambda w: f"{IDS[w[0]]}-{w[1][0]}x{w[1][1]}")
def test_many_rows(F, which, more):
    fmt, tile = which
    M, N, K = MANY[which]
    assert F.fp4q_selftest_gemm_fp8_choice(fmt, M, N + more, K) == tile + (1,)
    check(F, M, N + more, K, fmt, TYPES)
