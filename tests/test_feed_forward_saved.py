"""What the feed-forward block's backward refuses of what is said to be its forward's, on the CPU."""

import pytest
import torch

from dense_fp32_gemm_sm_gb300.feed_forward import FeedForward, Saved


def half(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("z,h", [(half(5, 6), half(4, 6)), (half(5, 6), half(5, 5)), (half(5, 6), half(5, 6).half()),
                                 (half(6, 5).t(), half(5, 6)), (half(5, 6), half(6, 5).t()), (half(5, 12)[:, :6], half(5, 6)),
                                 (half(30), half(5, 6))])
def test_pre_activations_and_hidden_values(z, h):
    with pytest.raises(ValueError):
        FeedForward(half(4, 6), half(6, 4)).backward(half(5, 4), Saved(half(5, 4), z, h, None))
