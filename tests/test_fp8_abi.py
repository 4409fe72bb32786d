"""Refusals of the 8-bit entry points, without a GPU: every argument error comes back as a status
before any CUDA call."""

import pytest

A = 1 << 20            # an aligned fake address: never dereferenced, validation fails first
FAR = [A + (i << 30) for i in range(1, 9)]


@pytest.fixture(scope="module")
def F():
    from microscaling_fp4_quantization_b200 import build
    build.build()
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


def test_quantize_refusals(F):
    def q(fmt=0, dtype=0, rows=1, x=A, ldx=256, M=4, K=256, codes=FAR[0], scales=FAR[1]):
        return F.raw_call("fp4q_quantize_fp8", fmt, dtype, rows, x, ldx, M, K, codes, scales, None)
    for bad in (dict(fmt=2), dict(fmt=-1), dict(dtype=2), dict(rows=64), dict(rows=0)):
        assert q(**bad) == F.FP4Q_ERR_UNSUPPORTED, bad
    for bad in (dict(K=200), dict(M=-1), dict(K=-16), dict(ldx=248), dict(ldx=260), dict(M=1 << 30), dict(K=1 << 31, ldx=1 << 31),
                dict(M=1 << 20, ldx=1 << 21)):
        assert q(**bad) == F.FP4Q_ERR_SHAPE, bad
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(codes=A), dict(codes=A + 512), dict(scales=A + 2044),
                dict(scales=FAR[0] + 1020)):
        assert q(**bad) == F.FP4Q_ERR_ARG, bad
    for bad in (dict(x=A + 8), dict(codes=A + 8), dict(scales=FAR[1] + 2)):
        assert q(**bad) == F.FP4Q_ERR_ALIGN, bad
    assert q(M=0, x=None, codes=None, scales=None) == F.FP4Q_OK
    assert q(K=0, x=None, codes=None, scales=None) == F.FP4Q_OK


def test_norm_refusals(F):
    def n(fmt=0, dtype=0, x=A, ldx=256, r=FAR[0], ldr=256, w=FAR[1], eps=1e-6, M=4, K=256, ro=FAR[2], ldo=256,
          codes=FAR[3], scales=FAR[4]):
        return F.raw_call("fp4q_add_rmsnorm_fp8", fmt, dtype, x, ldx, r, ldr, w, eps, M, K, ro, ldo, codes, scales, None)
    for bad in (dict(fmt=2), dict(dtype=2)):
        assert n(**bad) == F.FP4Q_ERR_UNSUPPORTED, bad
    for bad in (dict(K=200), dict(M=-1), dict(ldx=248), dict(ldr=252), dict(ldo=240),
                dict(K=32784, ldx=32784, ldr=32784, ldo=32784)):
        assert n(**bad) == F.FP4Q_ERR_SHAPE, bad
    for bad in (dict(x=None), dict(w=None), dict(codes=None), dict(scales=None), dict(r=None), dict(ro=None),
                dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(ro=A + 512), dict(ro=FAR[0] + 16), dict(ro=A, ldo=264), dict(ro=FAR[1]),
                dict(codes=A), dict(codes=FAR[0]), dict(codes=FAR[1]), dict(codes=FAR[2]), dict(scales=FAR[3]),
                dict(scales=A)):
        assert n(**bad) == F.FP4Q_ERR_ARG, bad
    for bad in (dict(x=A + 8), dict(r=FAR[0] + 8), dict(w=FAR[1] + 2), dict(ro=FAR[2] + 4), dict(codes=FAR[3] + 8),
                dict(scales=FAR[4] + 1)):
        assert n(**bad) == F.FP4Q_ERR_ALIGN, bad
    assert n(M=0, x=None, w=None, codes=None, scales=None) == F.FP4Q_OK


def test_arrays_between_each_others_rows_are_refused(F):
    """An array reaches from its first to its last byte: one in the gaps between another's rows overlaps it."""
    assert F.raw_call("fp4q_add_rmsnorm_fp8", 0, 0, A, 512, FAR[0], 256, FAR[1], 1e-6, 4, 256, A + 512, 512, FAR[3],
                      FAR[4], None) == F.FP4Q_ERR_ARG
    assert F.raw_call("fp4q_quantize_fp8", 0, 0, 1, A, 1024, 2, 256, A + 512, FAR[1], None) == F.FP4Q_ERR_ARG


def test_gemm_refusals(F):
    def g(fmt=0, dt=0, ac=A, sa=FAR[0], bc=FAR[1], sb=FAR[2], M=4, N=130, K=256, d=FAR[3]):
        return F.raw_call("fp4q_gemm_fp8", fmt, dt, ac, sa, bc, sb, M, N, K, d, None)
    for bad in (dict(fmt=2), dict(dt=3), dict(dt=-1)):
        assert g(**bad) == F.FP4Q_ERR_UNSUPPORTED, bad
    for bad in (dict(K=200), dict(K=0), dict(M=-1), dict(N=-1), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31),
                dict(M=1 << 30, N=1 << 30, K=16), dict(M=1 << 30, K=1 << 20)):
        assert g(**bad) == F.FP4Q_ERR_SHAPE, bad
    for bad in (dict(ac=None), dict(sa=None), dict(bc=None), dict(sb=None), dict(d=None), dict(d=A), dict(d=FAR[0]),
                dict(d=FAR[1] + 256), dict(d=FAR[2])):
        assert g(**bad) == F.FP4Q_ERR_ARG, bad
    for bad in (dict(ac=A + 8), dict(bc=FAR[1] + 8), dict(sa=FAR[0] + 2), dict(sb=FAR[2] + 1), dict(d=FAR[3] + 8)):
        assert g(**bad) == F.FP4Q_ERR_ALIGN, bad
    assert g(M=0, ac=None, sa=None, d=None) == F.FP4Q_OK
    assert g(N=0, bc=None, sb=None, d=None) == F.FP4Q_OK
