"""The MXFP4 layer as a user has it: forward, backward, decoding, training."""

import pytest
import torch

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def through(x):
    return torch.from_numpy(ref.through(x.double().cpu().numpy()))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K,N", [(1, 70, 33), (5, 256, 300), (200, 130, 257)])
@pytest.mark.parametrize("relu", [True, False])
def test_forward_backward_decode(M, K, N, relu, dt):
    from dense_fp32_gemm_sm_gb300.mxfp4_layer import Mxfp4Layer

    g = torch.Generator().manual_seed(M + N)
    w, x, go = (torch.randn(*s, generator=g).to(dt) for s in ((K, N), (M, K), (M, N)))
    b = torch.randn(N, generator=g)
    layer = Mxfp4Layer(w.cuda(), b.cuda(), relu)
    y = layer.forward(x.cuda())
    d = layer.decode(x.cuda())
    dx, dw, db = layer.backward(go.cuda(), y)
    # The definition in 64 bits.  FP32 sums of at most 300 terms are off by less than 300 * 2^-23
    # of the sum of magnitudes; rounding to the type adds 2^-8 at most of the value.
    u = {torch.float32: 2.0**-24, torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}[dt]

    def near(got, a, b_, add=None, gate=None):
        want, mag = a @ b_, a.abs() @ b_.abs()
        if add is not None:
            want, mag = want + add, mag + add.abs()
        if gate:
            want = want.clamp(min=0)
        assert ((got.double().cpu() - want).abs() <= 300 * 2.0**-23 * mag + u * want.abs() + 2.0**-25).all()

    near(y, through(x), through(w.t()).t(), b.double(), relu)
    near(d, through(x), through(w.t()).t(), b.double(), relu)
    gate = go.double() * (y.double().cpu() > 0) if relu else go.double()
    near(dx, through(gate), through(w).t())
    near(dw, through(x.t()), through(gate.t()).t())
    assert ((db.double().cpu() - gate.sum(0)).abs() <= M * 2.0**-23 * gate.abs().sum(0)).all()


def test_refusals_and_empty_batches():
    from dense_fp32_gemm_sm_gb300.mxfp4_layer import Mxfp4Layer

    w = torch.randn(64, 32, device="cuda")
    for bad in (w.double(), w.t(), w[0]):
        with pytest.raises(ValueError):
            Mxfp4Layer(bad)
    layer = Mxfp4Layer(w)
    for bad in (torch.zeros(3, 63, device="cuda"), torch.zeros(3, 64, device="cuda").half()):
        with pytest.raises(ValueError):
            layer.forward(bad)
        with pytest.raises(ValueError):
            layer.decode(bad)
    none = torch.empty(0, 64, device="cuda")
    assert layer.forward(none).shape == (0, 32) and layer.decode(none).shape == (0, 32)
    dx, dw, db = layer.backward(torch.empty(0, 32, device="cuda"), torch.empty(0, 32, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_training_lowers_the_loss():
    from dense_fp32_gemm_sm_gb300 import mxfp4_layer

    losses = mxfp4_layer.main(steps=60)
    # (4-bit gradients do not vanish at the optimum, so it does not reach 0)
    assert losses[-1] < 0.25 * losses[0]


def test_decoding_on_two_streams_at_once():
    from dense_fp32_gemm_sm_gb300.mxfp4_layer import Mxfp4Layer

    layer = Mxfp4Layer(torch.randn(1000, 520, device="cuda"))
    x = [torch.randn(40, 1000, device="cuda") for _ in range(2)]
    want = [layer.decode(v) for v in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(50):
        for s, v, out in zip(streams, x, got):
            with torch.cuda.stream(s):
                out.append(layer.decode(v))
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for w, ys in zip(want, got) for y in ys)
