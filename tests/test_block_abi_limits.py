"""Sizes that one launch of the gated block's gradient cannot take are refused on
the host: the runtime cuts a grid of 2^32 threads and more without an error.  No
GPU: a call that passes validation ends at the device check (status 4 or 5)."""
import pytest

from test_block_abi import FAKE, L  # noqa: F401


@pytest.mark.parametrize("inter", [32, 64, 14336, 1 << 21])
def test_glu_backward_rows_of_one_launch(L, inter):  # noqa: F811
    import torch
    most = ((1 << 34) - 1024) // inter
    call = lambda m: L.q3_glu_backward(FAKE, 2 * inter, FAKE, inter, 0, m, inter, FAKE, 2 * inter, None)  # noqa: E731
    for m in (most + 1, most + 2, 2 * most, (1 << 31) - 1):
        if m < 1 << 31:
            assert call(m) == 2, m
    if not torch.cuda.is_available():   # the largest one is past validation
        assert call(most) not in (0, 1, 2, 3)
