"""Quantizer and product back to back, without a wait of the host between them, through buffers of codes and
scales that every turn writes anew: each product reads the turn's own, though it may have started while they
were being written."""

import pytest
import torch

pytestmark = pytest.mark.gpu

TURNS = 24
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def F(cuda_device):
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


def values(rows, cols, seed):
    """Rows whose magnitudes, and so whose scales, change from seed to seed."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return (x * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda").float())).to(BF16)


@pytest.mark.parametrize("fmt", [0, 1], ids=["f32", "e8m0"])
@pytest.mark.parametrize("M,N", [(1, 2048), (24, 2048), (64, 2048), (200, 2048), (1100, 2048), (2500, 2056)])
def test_8bit(F, M, N, fmt):
    K = 1040
    b = F.quantize_fp8(values(N, K, 1000), 128, fmt)
    w = torch.ones(K, dtype=BF16, device="cuda")
    xs = [values(M, K, i) for i in range(TURNS)]
    want = []
    for i, x in enumerate(xs):
        c, s = F.quantize_fp8(x, 1, fmt) if i % 2 else F.add_rmsnorm_fp8(x, None, w, 1e-6, fmt)[:2]
        torch.cuda.synchronize()
        want.append(F.gemm_fp8(c, s, *b))
        torch.cuda.synchronize()
    codes, scales = torch.zeros_like(c), torch.zeros_like(s)
    got = [torch.empty_like(want[0]) for _ in xs]
    torch.cuda.synchronize()
    for i, x in enumerate(xs):
        if i % 2:
            F.quantize_fp8(x, 1, fmt, codes=codes, scales=scales)
        else:
            F.add_rmsnorm_fp8(x, None, w, 1e-6, fmt, codes=codes, scales=scales)
        F.gemm_fp8(codes, scales, *b, out=got[i])
    torch.cuda.synchronize()
    assert F.fp4q_device_status() == F.FP4Q_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N", [(1, 2048), (130, 2048), (1100, 2048), (2500, 2080)])
def test_fp4(F, M, N, fmt):
    K = 1024
    if fmt == "nvfp4":
        code, plan = F.FP4Q_NVFP4, F.fp4q_plan_create(F.FP4Q_NVFP4, 16, 16, F.FP4Q_SCALE_NV_DYNAMIC)
    else:
        code, plan = F.FP4Q_MXFP4, F.fp4q_plan_create(F.FP4Q_MXFP4, 32, 32, F.FP4Q_SCALE_FLOOR_OCP)
    b = F.rotate_quantize(plan, values(N, K, 1000))
    xs = [values(M, K, i) for i in range(TURNS)]
    want = []

    def product(a, out):
        F.fp4q_gemm(code, a[0], a[1], a[2], b[0], b[1], b[2], M, N, K, out)
        return out

    for x in xs:
        a = F.rotate_quantize(plan, x)
        torch.cuda.synchronize()
        want.append(product(a, torch.empty((M, N), dtype=BF16, device="cuda")))
        torch.cuda.synchronize()
    a = F.empty_outputs(plan, M, K)
    got = [torch.empty_like(want[0]) for _ in xs]
    torch.cuda.synchronize()
    for x, d in zip(xs, got):
        F.fp4q_rotate_quantize(plan, x, M, K, a[0], a[1], a[2] if code == F.FP4Q_NVFP4 else None)
        product(a, d)
    torch.cuda.synchronize()
    assert F.fp4q_device_status() == F.FP4Q_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)
