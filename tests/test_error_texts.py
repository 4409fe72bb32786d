"""What the status texts tell a caller of each family of calls (CPU)."""

import pytest


@pytest.fixture(scope="module")
def F():
    from microscaling_fp4_quantization_b200 import build
    build.build()
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


def test_shape_text_names_each_rule_for_k(F):
    text = F.fp4q_status_string(F.FP4Q_ERR_SHAPE)
    assert "max(group, hadamard_block)" in text          # the FP4 calls'
    assert "256 in fp4q_gemm" in text and "16 in the 8-bit calls" in text


def test_alignment_text_names_the_tensor_scale_and_the_scales(F):
    text = F.fp4q_status_string(F.FP4Q_ERR_ALIGN)
    assert "16 bytes for arrays" in text and "tensor scale" in text and "fp32 scales" in text
