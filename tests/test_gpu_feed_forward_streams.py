"""The feed-forward block's backward on another stream than its forward."""

import pytest
import torch

from test_gpu_feed_forward import block
from test_gpu_gemm16 import _cuda  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [None, 3])
def test_what_the_forward_left_stays_until_it_is_read(E):
    """The backward waits on its stream while what it reads is dropped, and the memory filled on the forward's."""
    M, K, N = 2048, 512, 1024
    ff, _, g = block(K, N, E, torch.bfloat16, "gelu", True, True)
    gr = torch.randn(M, K, generator=g).bfloat16().cuda()
    x0 = torch.randn(M, K, generator=g).bfloat16().cuda()
    offsets = None if E is None else torch.tensor([0, 700, 700, M], dtype=torch.int32).cuda()
    y, saved = ff.forward(x0, offsets)
    want = (y, *ff.backward(gr, saved))
    torch.cuda._sleep(1)  # (kernels are loaded at their first launch, and wait for the GPU then)
    torch.full((8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    del y, saved
    side = torch.cuda.Stream()
    x = x0.clone()
    y, saved = ff.forward(x, offsets)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # 50 ms
        got = ff.backward(gr, saved)
    del saved, x
    filled = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for shape in ((M, N), (M, K)) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, *got), want))
    del filled


def test_captured_on_two_streams():
    """Forward and backward on two streams of one capture, replayed."""
    M, K, N = 300, 128, 256
    ff, _, g = block(K, N, None, torch.bfloat16, "silu", True, False)
    x, gr = (torch.randn(M, K, generator=g).bfloat16().cuda() for _ in range(2))
    y, saved = ff.forward(x)
    want = (y, *ff.backward(gr, saved))
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        y, saved = ff.forward(x)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            got = ff.backward(gr, saved)
        main.wait_stream(side)
        del saved
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, *got), want))
