"""What the feed-forward block refuses, on the CPU: nothing is launched."""

import pytest
import torch

from dense_fp32_gemm_sm_gb300.feed_forward import FeedForward, Saved


def half(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("w1,w2", [
    (torch.zeros(4, 6), torch.zeros(6, 4)), (half(4), half(4)), (half(4, 6), half(4, 6)), (half(4, 6), half(6, 4).half()),
    (half(2, 4, 6), half(6, 4)), (half(2, 4, 6), half(3, 6, 4)), (half(6, 4).t(), half(6, 4)), (half(4, 6), half(4, 6).t()),
])
def test_weights(w1, w2):
    with pytest.raises(ValueError):
        FeedForward(w1, w2)


@pytest.mark.parametrize("kw", [dict(b1=half(6)), dict(b1=torch.zeros(4)), dict(b2=torch.zeros(6)), dict(b2=torch.zeros(8)[::2]),
                                dict(act="tanh"), dict(grad_type=torch.float16), dict(b1=torch.zeros(1, 6))])
def test_options(kw):
    with pytest.raises(ValueError):
        FeedForward(half(4, 6), half(6, 4), **kw)


def test_tokens_and_offsets():
    one, experts = FeedForward(half(4, 6), half(6, 4)), FeedForward(half(2, 4, 6), half(2, 6, 4))
    off = torch.zeros(3, dtype=torch.int32)
    for x in (torch.zeros(5, 4), half(5, 6), half(5), half(4, 5).t(), half(1, 4).expand(5, 4)):
        with pytest.raises(ValueError):
            one.forward(x)
        with pytest.raises(ValueError):
            experts(x, off)
    with pytest.raises(ValueError):
        one.forward(half(5, 4), off)
    for bad in (None, off.long(), off[:2], torch.zeros(6, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            experts.forward(half(5, 4), bad)
    with pytest.raises(ValueError):
        one.backward(half(5, 4), Saved(half(6, 4), half(6, 6), half(6, 6), None))
    for saved in (Saved(half(5, 4), half(5, 8), half(5, 8), None), Saved(half(5, 3), half(5, 6), half(5, 6), None),
                  Saved(half(5, 4), half(4, 6), half(4, 6), None), Saved(half(5, 4), half(5, 6), half(5, 6), off),
                  Saved(half(5, 4), half(5, 6).half(), half(5, 6), None)):
        with pytest.raises(ValueError):
            one.backward(half(5, 4), saved)
    with pytest.raises(ValueError):
        experts.backward(half(5, 4), Saved(half(5, 4), half(5, 6), half(5, 6), None))


def test_rows_of_one_column():
    assert FeedForward(half(1, 6), half(6, 1))._rows(half(1, 5).t(), 1) == 1
