"""The differentiable calls say that autograd does not record them, and which call
gives the gradient.  No GPU."""
import pytest


@pytest.mark.parametrize("name,backward", [("q3_gemm", "q3_gemm_backward"), ("q3_glu", "q3_glu_backward"),
                                           ("q3_residual_norm", "q3_residual_norm_backward"), ("q3_ffn", None)])
def test_autograd_is_named_at_the_call(name, backward):
    from bit_fp8_codebook_amd import _block
    said = " ".join(getattr(_block, name).__doc__.split())
    assert "recorded by autograd" in said
    if backward:
        assert backward in said and callable(getattr(_block, backward))
