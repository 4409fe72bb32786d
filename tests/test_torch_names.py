"""The tensor calls on a torch that lacks what they would rather use: a private name for the current stream,
and the E8M0 type (only float32 scales are then offered)."""

import pytest
import torch


@pytest.fixture
def F(monkeypatch):
    from microscaling_fp4_quantization_b200 import build
    build.build()
    from microscaling_fp4_quantization_b200 import fp4q
    for name in ("_torch", "_e4m3", "_raw_stream", "_current_device"):
        monkeypatch.setattr(fp4q, name, None)
    for name in ("_fp8_in_dtypes", "_fp8_out_dtypes", "_fp8_scale_dtypes"):
        monkeypatch.setattr(fp4q, name, {})
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch, "float8_e8m0fnu", raising=False)
    fp4q._fp8_init()
    return fp4q


def test_the_current_stream_by_public_names(F, monkeypatch):
    class Stream:
        cuda_stream = 77
    asked = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: (asked.append(device), Stream)[1])
    assert F._raw_stream(3) == 77 and asked == [3]


def test_float32_scales_without_the_e8m0_type(F):
    assert F._fp8_scale_dtypes == {F.FP4Q_FP8_SCALE_F32: torch.float32}


@pytest.mark.gpu
def test_calls_and_refusals(F, cuda_device):
    x = torch.randn((20, 256), device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c, s = F.quantize_fp8(x)
        b = F.quantize_fp8(x, 128)
        d = F.gemm_fp8(c, s, *b)
        _, _, stored = F.add_rmsnorm_fp8(x, x, x[0], 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(stored, x + x)
    from test_fp8 import check_gemm
    check_gemm(d, (c, s), b, 256)
    with pytest.raises(ValueError):
        F.quantize_fp8(x, 1, F.FP4Q_FP8_SCALE_E8M0)
    with pytest.raises(ValueError):
        F.add_rmsnorm_fp8(x, None, x[0], 1e-6, F.FP4Q_FP8_SCALE_E8M0)
    with pytest.raises(ValueError):
        F.gemm_fp8(c, s.half(), *b)
