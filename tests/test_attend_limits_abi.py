"""Where the arguments of the attention sublayer's and the log probabilities' entry
points end, without a GPU: refusals before any HIP call."""
import pytest

from test_attend_abi import _batch, _cache, _ref
from test_block_abi import FAKE, L  # noqa: F401


@pytest.mark.parametrize("t", [4.23e-39, 3e-39, 2.95e-39, 1e-45])
def test_temperatures_too_cold(L, t):  # noqa: F811
    # 1 / t is still finite in fp32 down to 2.94e-39, log2(e) / t only to 4.24e-39
    assert L.q3_logprobs(FAKE, 2, 100, 100, FAKE, t, 0, FAKE, None, None, None, None, None, 0, None) == 1
    assert L.q3_logprobs_backward(FAKE, 2, 100, 100, FAKE, t, FAKE, FAKE, None, FAKE + 4096, 100, 1, None) == 1


@pytest.mark.parametrize("scale", [2.36e38, -2.36e38, 3.4e38])
def test_scales_too_large(L, scale):  # noqa: F811
    # scale is finite in fp32 up to 3.4e38, scale log2(e) only to 2.35e38
    assert L.q3_paged_attention(FAKE, 256, 4, _ref(_cache()), _ref(_batch()), scale, 0, FAKE, 256, FAKE, 3, FAKE,
                                1 << 40, None) == 1


@pytest.mark.parametrize("window", [-1, 1 << 31, (1 << 32) + 5, 1 << 40])
def test_the_binding_takes_no_window_past_32_bits(window):
    # as an int32 the last two would be windows of 5 and of 0, which is none at all
    import torch
    from bit_fp8_codebook_amd import _block as b
    with pytest.raises(ValueError, match="window"):
        b.q3_paged_attention(torch.zeros(3, 256, dtype=torch.bfloat16), None, None, window=window)
