"""Several forwards of the MXFP4 layer before their backwards: the gradients are those of each forward
followed by its own backward, bit for bit."""

import pytest
import torch

pytestmark = pytest.mark.gpu

K, N = 130, 257


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def steps(sizes, dt, relu):
    from dense_fp32_gemm_sm_gb300.mxfp4_layer import Mxfp4Layer

    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    layer = Mxfp4Layer(rand(K, N).to(dt), rand(N), relu)
    data = [(rand(M, K).to(dt), rand(M, N).to(dt)) for M in sizes]
    want = []
    for x, go in data:
        y = layer.forward(x)
        want.append((y, *layer.backward(go, y)))
    return layer, data, want


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("relu", [True, False])
def test_forwards_of_one_size(dt, relu):
    layer, data, want = steps((70, 70, 33, 70, 70), dt, relu)
    kept = []
    for x, _ in data:
        kept.append((layer.forward(x), layer.saved))
    layer.forward(torch.zeros_like(data[0][0]))  # an evaluation in between takes nothing from them
    for (y, saved), (_, go), w in reversed(list(zip(kept, data, want))):
        assert same((y, *layer.backward(go, y.clone(), saved)), w)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_forwards_of_a_few_sizes(dt):
    layer, data, want = steps((5, 70, 33, 200), dt, True)
    outs = [layer.forward(x) for x, _ in data]
    for y, (_, go), w in zip(outs, data, want):
        assert same((y, *layer.backward(go, y)), w)
    layer.forward(data[0][0][:3].contiguous())  # a fifth size: the oldest tokens go
    for y, (_, go), w in list(zip(outs, data, want))[1:]:
        assert same((y, *layer.backward(go, y)), w)
    with pytest.raises(ValueError):
        layer.backward(data[0][1], outs[0])
