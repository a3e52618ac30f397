"""Quantising on every way that a tile can reach a CTA, with many tiles for each CTA, against the
definition: rows on 16 bytes, on 4 and on neither, with and without ReLU's gate.

A CTA walks over tiles of 128 x 128 (at most three CTAs an SM do), its copies, gates and loads of the next
tiles under way in a ring of stages.  Narrow or flat matrices have many tiles for little data, and no
two tiles hold the same."""

import numpy as np
import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": (fg.F32, torch.float32), "bf16": (fg.BF16, torch.bfloat16), "f16": (fg.F16, torch.float16)}
SENTINEL = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    fg.library()


def on_gpu(x, dt, ld):
    """x with leading dimension ld, NaN between the rows: its tensor, and its values in float64."""
    buf = torch.full((x.shape[0], ld), float("nan"), dtype=dt)
    buf[:, :x.shape[1]] = torch.from_numpy(x).to(dt)
    return buf.cuda(), buf[:, :x.shape[1]].double().numpy()


def leading(N, dt, align):
    """The least leading dimension above N whose rows start on `align` bytes and on no more (0: on an element)."""
    es = torch.empty(0, dtype=dt).element_size()
    return next(ld for ld in range(N + 1, N + 65) if ld * es % align == 0 and (align == 16 or ld * es % (2 * align)))


class Quantised:
    def __init__(self, rows, cols):
        self.shape, self.ld = (rows, cols), 16 * ref.blocks(cols) + 16
        self.codes = torch.full((rows, self.ld), SENTINEL, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((fg.mxfp4_scales_size(rows, cols),), SENTINEL, dtype=torch.uint8, device="cuda")

    @property
    def args(self):
        return self.codes, self.ld, self.scales

    def check(self, want):
        assert want.shape == self.shape
        parts = [ref.encode(want[i:i + 16384]) for i in range(0, len(want), 16384)]  # (rows are independent)
        code, s = (np.concatenate(p) for p in zip(*parts))
        assert np.array_equal(self.codes.cpu().numpy(), ref.pack_codes(code, self.ld, SENTINEL))
        assert np.array_equal(self.scales.cpu().numpy(), ref.pack_scales(s))


def values(rng, M, N):
    x = rng.standard_normal((M, N)) * np.exp2(rng.integers(-6, 6, (M, 1)))
    kind = rng.random((M, N))
    x[kind < 0.1] = 0
    x[kind > 0.98] *= 30
    return x


# (ragged at both ends; aligned rows of 24 elements, and two columns or rows of tiles)
SHAPES = [(130, 264), (128 * 3 + 8, 128 * 2), (128 * 920 + 5, 24), (12, 128 * 920 + 8), (128 * 320, 136)]
ALIGNMENTS = {"f32": (16, 4), "bf16": (16, 4, 2), "f16": (16, 4, 2)}
WAYS = [(t, a) for t in TYPES for a in ALIGNMENTS[t]]


@pytest.mark.parametrize("gate,M,N", [(True, *s) for s in SHAPES] + [(False, *s) for s in SHAPES[:-1]])
@pytest.mark.parametrize("t,align", WAYS)
def test_gradient(t, align, gate, M, N):
    type_, dt = TYPES[t]
    rng = np.random.default_rng(M + N + align)
    g = values(rng, M, N)
    y = np.maximum(rng.standard_normal((M, N)), 0)
    y[rng.random((M, N)) < 0.01] = np.nan  # not greater than 0
    if gate:
        closed = ~(y > 0)
        g[closed & (rng.random((M, N)) < 0.1)] = np.nan  # behind a closed gate nothing matters
    ld = leading(N, dt, align)
    G, g = on_gpu(g, dt, ld)
    Y, y = on_gpu(y, dt, ld)
    assert G.data_ptr() % 16 == 0 and Y.data_ptr() % 16 == 0
    if gate:
        g = np.where(y > 0, g, 0)
    r, c = Quantised(M, N), Quantised(N, M)
    ws = torch.full((fg.mxfp4_quantize_grad_workspace_size(M, N),), 0xFF, dtype=torch.uint8, device="cuda")
    bias = torch.full((N,), float("nan"), device="cuda")
    fg.mxfp4_quantize_grad(type_, M, N, G, ld, Y if gate else None, ld, *r.args, *c.args, bias, ws, ws.numel())
    torch.cuda.synchronize()
    r.check(g)
    c.check(g.T)
    # any order of FP32 additions: each of at most M - 1 is off by 2^-24 of a sum of at most sum |g|
    err = np.abs(bias.cpu().numpy().astype(np.float64) - g.sum(0))
    assert (err <= (M - 1) * 2.0**-24 * np.abs(g).sum(0)).all()


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("t,align", WAYS)
def test_both_directions(t, align, M, N):
    type_, dt = TYPES[t]
    ld = leading(N, dt, align)
    X, x = on_gpu(values(np.random.default_rng(M * align + N), M, N), dt, ld)
    r, c = Quantised(M, N), Quantised(N, M)
    fg.mxfp4_quantize(type_, M, N, X, ld, *r.args, *c.args)
    torch.cuda.synchronize()
    r.check(x)
    c.check(x.T)


def test_a_cta_has_several_tiles():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert [-(-M // 128) * -(-N // 128) // (3 * sms) for M, N in SHAPES] >= [0, 0, 2, 2, 1]
