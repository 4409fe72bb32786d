"""The residual RMS norm at the ends of fp32's range: the values of eps it takes, and rows whose squares fp32
does not hold."""

import numpy as np
import pytest


@pytest.fixture(scope="module")
def lib():
    from microscaling_fp4_quantization_b200 import build
    build.build()
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


def test_every_finite_eps_is_taken(lib):
    def n(eps):   # an empty x: refused for its eps or not at all
        return lib.raw_call("fp4q_add_rmsnorm_fp8", 0, 0, None, 256, None, 0, None, eps, 0, 256, None, 0, None, None, None)
    top = float(np.finfo(np.float32).max)
    for eps in (0.0, 2.0 ** -149, 1e-6, 3.1e38, top):
        assert n(eps) == lib.FP4Q_OK, eps
    for eps in (-2.0 ** -149, float("nan"), float("inf"), float("-inf"), 1e39):
        assert n(eps) == lib.FP4Q_ERR_ARG, eps


@pytest.mark.gpu
def test_rows_of_tiny_values(cuda_device):
    """Squares that fp32 does not hold: NaN without eps; with it, y = h / sqrt(eps) like any other row (the
    codes' magnitudes, which one factor for the row leaves alone, come out as the values', in steps of E4M3)."""
    import torch

    from microscaling_fp4_quantization_b200 import fp4q as F
    from oracle import fp8_oracle as o
    K = 512
    h = np.tile(np.array([1.0, -0.5, 0.25, 0.0], np.float32), K // 4)
    x = torch.from_numpy(np.stack([h * 2.0 ** -80, h, h * 2.0 ** -70])).to(torch.bfloat16).cuda()
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    codes, scales, _ = F.add_rmsnorm_fp8(x, None, w, 0.0)
    torch.cuda.synchronize()
    s = scales.cpu().numpy()
    assert np.all(np.isnan(s[0])) and np.all(np.isfinite(s[1:]))
    codes, scales, _ = F.add_rmsnorm_fp8(x, None, w, 2.0 ** -40)
    torch.cuda.synchronize()
    v = o.operand(codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), 1)
    # sqrt(2^-40) = 2^-20: exact factors, maxima 2^-60 and 2^-50; the codes 448, -224, 112 and 0 are exact, and the
    # scale is a quotient by 448, rounded once
    for row, top in ((0, 2.0 ** -60), (2, 2.0 ** -50)):
        assert np.all(np.abs(v[row] - h * top) <= 2.0 ** -24 * top)
