"""Quantising to MXFP4 and back, on the GPU, against the definition in 64 bits.

Codes and scales are whole numbers: every byte has to be equal, those of the padding (the last
block's absent elements, the scale atoms' absent rows and blocks) included, and nothing else
may be written.  Dequantised values are exact in every type but where the type cannot hold
them (rounded once).  The bias's gradient is a sum of FP32 numbers in some fixed order: it
lies within (M - 1) * 2^-24 * sum |g| of the exact sum.
"""

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


def on_gpu(x, dt, pad=0, offset=0, fill=float("nan")):
    """x on the GPU with `pad` elements between its rows, `offset` elements past an aligned
    address: (tensor that owns it, address, leading dimension, the values in float64)."""
    rows, cols = x.shape
    ld = cols + pad
    buf = torch.full((rows * ld + offset + 8,), fill, dtype=dt)
    v = buf[offset:offset + rows * ld].view(rows, ld)
    v[:, :cols] = torch.from_numpy(np.asarray(x)).to(dt)
    dev = buf.cuda()
    return dev, dev.data_ptr() + offset * dev.element_size(), ld, v[:, :cols].double().numpy()


class Quantised:
    """Room for a rows x cols quantised matrix, filled with a sentinel."""

    def __init__(self, rows, cols, extra=0):
        self.rows, self.cols = rows, cols
        self.ld = 16 * ref.blocks(cols) + extra
        self.codes = torch.full((rows, self.ld), SENTINEL, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((fg.mxfp4_scales_size(rows, cols) + 16,), SENTINEL, dtype=torch.uint8,
                                 device="cuda")

    @property
    def args(self):
        return self.codes, self.ld, self.scales

    def check(self, want):
        code, s = ref.encode(want)
        got = self.codes.cpu().numpy()
        assert np.array_equal(got, ref.pack_codes(code, self.ld, SENTINEL))
        got = self.scales.cpu().numpy()
        assert np.array_equal(got[:-16], ref.pack_scales(s)) and (got[-16:] == SENTINEL).all()


def draw(rng, M, N):
    """Blocks of many magnitudes, with zeros, loud elements and halfway cases among them."""
    x = rng.standard_normal((M, N)) * np.exp2(rng.integers(-12, 6, (M, 1)))
    kind = rng.random((M, N))
    x[kind < 0.1] = 0
    x[kind > 0.97] *= 30
    pick = (kind > 0.6) & (kind < 0.8)
    x[pick] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7, -0.25, -5, -2.5, 4, 8], pick.sum())
    return x


SHAPES = [(1, 1), (1, 32), (3, 33), (31, 127), (128, 128), (129, 257), (300, 40), (77, 1000), (260, 513)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("t", TYPES)
def test_both_directions(t, M, N):
    code, dt = TYPES[t]
    _, ptr, ld, x = hold = on_gpu(draw(np.random.default_rng(M * 1000 + N), M, N), dt)
    r, c = Quantised(M, N), Quantised(N, M, extra=16)
    fg.mxfp4_quantize(code, M, N, ptr, ld, r.codes, r.ld, r.scales, c.codes, c.ld, c.scales)
    torch.cuda.synchronize()
    r.check(x)
    c.check(x.T)
    del hold


@pytest.mark.parametrize("way", ["rows", "cols"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (8, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("t", TYPES)
def test_one_direction_any_alignment(t, pad, offset, way):
    code, dt = TYPES[t]
    M, N = 150, 320
    _, ptr, ld, x = hold = on_gpu(draw(np.random.default_rng(pad * 10 + offset), M, N), dt, pad, offset)
    q = Quantised(M, N, extra=32) if way == "rows" else Quantised(N, M)
    none = (None, 0, None)
    fg.mxfp4_quantize(code, M, N, ptr, ld, *(q.args + none if way == "rows" else none + q.args))
    torch.cuda.synchronize()
    q.check(x if way == "rows" else x.T)
    del hold


def test_special_values():
    x = np.zeros((40, 70))
    x[0, 0], x[1, 40], x[2, 69], x[3, 1] = np.nan, np.inf, -np.inf, -0.0
    x[4, :3] = 2.0**-149, -2.0**-130, 2.0**-126  # subnormals: the scale ends at 2^-127
    x[5, :2] = 3.4e38, -1.0e-30
    x[6, :2] = 2.0**127, 2.0**125
    x[7, 33:35] = 2.0**-149, 2.0**-148
    x[8, :2] = 7.0 * 2.0**-127, 1.5 * 2.0**-124
    _, ptr, ld, v = hold = on_gpu(x, torch.float32)
    r, c = Quantised(40, 70), Quantised(70, 40)
    fg.mxfp4_quantize(fg.F32, 40, 70, ptr, ld, r.codes, r.ld, r.scales, c.codes, c.ld, c.scales)
    torch.cuda.synchronize()
    r.check(v)
    c.check(v.T)
    del hold


def test_halves_keep_their_own_largest():
    # f16's largest and smallest magnitudes, bf16's subnormals
    x = np.array([[65504.0, -65504.0, 2.0**-24, 0.0] * 10])
    _, ptr, ld, v = hold = on_gpu(x, torch.float16)
    r = Quantised(1, 40)
    fg.mxfp4_quantize(fg.F16, 1, 40, ptr, ld, r.codes, r.ld, r.scales, None, 0, None)
    torch.cuda.synchronize()
    r.check(v)
    x = np.array([[2.0**-133, -2.0**-131, 0.0, 0.0] * 10])
    _, ptr, ld, v = hold = on_gpu(x, torch.bfloat16)
    r = Quantised(1, 40)
    fg.mxfp4_quantize(fg.BF16, 1, 40, ptr, ld, r.codes, r.ld, r.scales, None, 0, None)
    torch.cuda.synchronize()
    r.check(v)
    del hold


@pytest.mark.parametrize("M,N", [(1, 1), (5, 33), (128, 64), (130, 257), (600, 200), (1, 4097)])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("t", TYPES)
def test_gradient_with_gate_and_bias(t, gate, M, N):
    code, dt = TYPES[t]
    rng = np.random.default_rng(M + N)
    g = draw(rng, M, N)
    y = np.maximum(rng.standard_normal((M, N)), 0)
    y[rng.random((M, N)) < 0.02] = np.nan  # not greater than 0: a closed gate
    if gate:
        g[(y <= 0) & (rng.random((M, N)) < 0.3)] = np.nan  # behind a closed gate nothing matters
        g[(y <= 0) & (rng.random((M, N)) < 0.3)] = np.inf
        y[0, 0] = 2.0**-20  # a small output is still an open gate
        g[0, 0] = 1.0
    _, gp, ldg, g = hold = on_gpu(g, dt, pad=1)
    _, yp, ldy, y = hold2 = on_gpu(y, dt, pad=2)
    if gate:
        g = np.where(y > 0, g, 0)
    r, c = Quantised(M, N), Quantised(N, M)
    ws = torch.full((max(16, fg.mxfp4_quantize_grad_workspace_size(M, N)),), 0xFF, dtype=torch.uint8, device="cuda")
    bias = torch.full((N,), float("nan"), device="cuda")
    fg.mxfp4_quantize_grad(code, M, N, gp, ldg, yp if gate else None, ldy if gate else 0, r.codes, r.ld, r.scales,
                           c.codes, c.ld, c.scales, bias, ws, ws.numel())
    torch.cuda.synchronize()
    r.check(g)
    c.check(g.T)
    err = np.abs(bias.cpu().numpy().astype(np.float64) - g.sum(0))
    assert (err <= (M - 1) * 2.0**-24 * np.abs(g).sum(0) + 1e-45).all()
    again = torch.empty_like(bias)
    fg.mxfp4_quantize_grad(code, M, N, gp, ldg, yp if gate else None, ldy if gate else 0, r.codes, r.ld, r.scales,
                           None, 0, None, again, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(bias, again)
    del hold, hold2


def test_gradient_is_the_bias_gradient_of_the_layer():
    # differences: the layer's output summed against G changes by h * bias_grad when its bias does
    rng = np.random.default_rng(3)
    M, N, h = 50, 40, 2.0**-8
    pre, G = rng.integers(-8, 9, (M, N)) + 0.5, rng.integers(-4, 5, (M, N)).astype(float)
    loss = lambda b: (np.maximum(pre + b, 0) * G).sum()  # noqa: E731
    _, gp, ldg, _ = hold = on_gpu(G, torch.float32)
    _, yp, ldy, _ = hold2 = on_gpu(np.maximum(pre, 0), torch.float32)
    r = Quantised(M, N)
    bias, ws = torch.empty(N, device="cuda"), torch.empty(4 * N, dtype=torch.uint8, device="cuda")
    fg.mxfp4_quantize_grad(fg.F32, M, N, gp, ldg, yp, ldy, r.codes, r.ld, r.scales, None, 0, None, bias, ws, 4 * N)
    got = bias.cpu().numpy()
    for j in range(N):
        d = np.zeros(N)
        d[j] = h
        assert got[j] == (loss(d) - loss(-d)) / (2 * h)
    del hold, hold2


def test_no_rows_give_a_zero_bias_gradient():
    bias = torch.full((33,), 5.0, device="cuda")
    fg.mxfp4_quantize_grad(fg.F32, 0, 33, None, 33, None, 0, None, 0, None, None, 0, None, bias, None, 0)
    torch.cuda.synchronize()
    assert not bias.any()


@pytest.mark.parametrize("M,N", [(1, 1), (3, 33), (129, 130), (50, 1024)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (8, 0), (0, 3)])
@pytest.mark.parametrize("t", TYPES)
def test_dequantize(t, M, N, pad, offset):
    code, dt = TYPES[t]
    rng = np.random.default_rng(N)
    c, s = ref.random_codes(rng, M, N, 115, 140)
    s[0, 0], s[-1, -1] = 0, 254
    if M > 2:
        s[2, 0] = 255
    codes = torch.from_numpy(ref.pack_codes(c, 16 * ref.blocks(N) + 16, 0x77)).cuda()
    scales = torch.from_numpy(ref.pack_scales(s)).cuda()
    ld = N + pad
    out = torch.full((M * ld + offset + 8,), -3.0, dtype=dt, device="cuda")
    fg.mxfp4_dequantize(code, M, N, codes, codes.shape[1], scales, out.data_ptr() + offset * out.element_size(), ld)
    torch.cuda.synchronize()
    want = torch.full_like(out, -3.0, device="cpu")
    want[offset:offset + M * ld].view(M, ld)[:, :N] = torch.from_numpy(ref.values(c, s)).float().to(dt)
    assert torch.equal(out.cpu().nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0))


def test_on_another_stream_after_its_producer():
    # the input is produced on the stream the call is given, so it must run behind it there
    stream = torch.cuda.Stream()
    x = torch.zeros(2000, 4096, device="cuda")
    r = Quantised(2000, 4096)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(20):
            x.add_(1.0)
        fg.mxfp4_quantize(fg.F32, 2000, 4096, x, 4096, r.codes, r.ld, r.scales, None, 0, None, stream=stream)
    stream.synchronize()
    # 20 = 1.25 * 2^4: scale 2^2, 5 is halfway between 4 and 6: the even code, 4
    assert (r.codes == 0x66).all() and set(r.scales[:-16].unique().tolist()) == {129, 0}


@pytest.mark.parametrize("M,N", [(5_000_001, 3), (2, 4_000_033)])
def test_very_tall_and_very_wide(M, N):
    # more rows than a grid dimension holds CTAs, and as many columns; every row (or column of
    # 32) repeats one of a few
    rng = np.random.default_rng(9)
    if M > N:
        pool = draw(rng, 64, N)  # (a column's blocks repeat every 64 rows)
        x = torch.from_numpy(pool).float().cuda()[torch.arange(M, device="cuda") % 64]
        r, c = Quantised(M, N), Quantised(N, M)
        fg.mxfp4_quantize(fg.F32, M, N, x, N, r.codes, r.ld, r.scales, c.codes, c.ld, c.scales)
        back, back_t = torch.empty_like(x), torch.empty(N, M, device="cuda")
        fg.mxfp4_dequantize(fg.F32, M, N, r.codes, r.ld, r.scales, back, N)
        fg.mxfp4_dequantize(fg.F32, N, M, c.codes, c.ld, c.scales, back_t, M)
        pool = x[:64].double().cpu().numpy()
        want = torch.from_numpy(ref.through(pool)).float().cuda()
        assert torch.equal(back, want[torch.arange(M, device="cuda") % 64])
        whole = torch.from_numpy(ref.through(np.concatenate([pool, pool[:M % 64]]).T)).float().cuda()
        full = M // 64 * 64
        assert torch.equal(back_t[:, :full].view(N, -1, 64), whole[:, None, :64].expand(N, full // 64, 64))
        tail = torch.from_numpy(ref.through(pool[:M % 64].T)).float().cuda()
        assert torch.equal(back_t[:, full:], tail)
    else:
        _, ptr, ld, x = hold = on_gpu(draw(rng, M, N), torch.float32)
        r, c = Quantised(M, N), Quantised(N, M)
        fg.mxfp4_quantize(fg.F32, M, N, ptr, ld, r.codes, r.ld, r.scales, c.codes, c.ld, c.scales)
        torch.cuda.synchronize()
        r.check(x)
        back = torch.empty(N, M, device="cuda")
        fg.mxfp4_dequantize(fg.F32, N, M, c.codes, c.ld, c.scales, back, M)
        pick = rng.integers(0, N, 2000)
        assert np.array_equal(back.cpu().numpy()[pick], ref.through(x.T[pick]))
        del hold


def test_offsets_beyond_32_bits():
    # more than 2^31 elements, and codes at byte offsets beyond 2^31
    M, N = 2**31 // 8192 + 129, 16384
    rows = torch.randn(7, N, device="cuda").to(torch.bfloat16)
    x = rows[torch.arange(M, device="cuda") % 7]
    r, c = Quantised(M, N), Quantised(N, M)
    fg.mxfp4_quantize(fg.BF16, M, N, x, N, r.codes, r.ld, r.scales, c.codes, c.ld, c.scales)
    torch.cuda.synchronize()
    code, s = ref.encode(rows.double().cpu().numpy())
    want = torch.from_numpy(ref.pack_codes(code)).cuda()
    for i in range(0, M, 65536):
        assert torch.equal(r.codes[i:i + 65536], want[torch.arange(i, min(M, i + 65536), device="cuda") % 7])
    back = torch.empty_like(x)
    fg.mxfp4_dequantize(fg.BF16, M, N, r.codes, r.ld, r.scales, back, N)
    want = torch.from_numpy(ref.values(code, s)).cuda().to(torch.bfloat16)
    for i in range(0, M, 65536):
        assert torch.equal(back[i:i + 65536], want[torch.arange(i, min(M, i + 65536), device="cuda") % 7])
    del back
    # columns: the last three, at the far end of the codes
    code, s = ref.encode(x[:, -3:].double().cpu().numpy().T)
    assert np.array_equal(c.codes[-3:].cpu().numpy(), ref.pack_codes(code))
    back = torch.empty(N, M, dtype=torch.bfloat16, device="cuda")
    fg.mxfp4_dequantize(fg.BF16, N, M, c.codes, c.ld, c.scales, back, M)
    assert torch.equal(back[-3:].cpu(), torch.from_numpy(ref.values(code, s)).to(torch.bfloat16))
