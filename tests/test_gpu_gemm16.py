"""16-bit products with a layer's epilogue on the GPU against 64 bits (tolerances: gemm16_ref)."""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import gemm16_ref as ref

pytestmark = pytest.mark.gpu

CODE = {"f32": fg.F32, "bf16": fg.BF16, "f16": fg.F16}
ACT = {"none": fg.ACT_NONE, "relu": fg.ACT_RELU, "gelu": fg.ACT_GELU, "silu": fg.ACT_SILU}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    fg.library()
    fg.device_status(clear=True)
    yield
    assert fg.device_status() == fg.OK


def values(g, rows, cols, dtype, ints=False, scale=1.0):
    if ints:
        return torch.randint(-3, 4, (rows, cols), generator=g).to(dtype)
    return (scale * torch.randn(rows, cols, generator=g)).to(dtype)


def product(t, M, N, K, out=None, ta=False, tb=False, alpha=1.0, bias=False, act="none", keep=False, beta=0.0, alias=False,
            grad=False, sums=False, pads=(0, 0, 0, 0, 0), offsets=(0, 0, 0, 0, 0), ints=False, seed=0, stream=None):
    """pads, offsets: of A, B, Z, R, Y."""
    g = torch.Generator().manual_seed(seed)
    dt, ot = ref.TYPES[t], ref.TYPES[out or t]
    a, b = values(g, M, K, dt, ints), values(g, K, N, dt, ints, max(K, 1) ** -0.5)
    A = ref.Buffer(a.t() if ta else a, pads[0], offsets[0])
    B = ref.Buffer(b.t() if tb else b, pads[1], offsets[1])
    bi = (torch.randint(-8, 9, (N,), generator=g) / 4.0) if bias else None
    r = values(g, M, N, ot, ints)
    z = values(g, M, N, dt)
    size = fg.gemm16_copy_workspace_size(ta, tb, 1, M, N, K) + fg.gemm16_sums_workspace_size(1, M, N)
    ws = torch.full((size,), 255, dtype=torch.uint8).cuda()
    common = (CODE[t], CODE[out or t], ta, tb, M, N, K, alpha, A.ptr, A.ld, B.ptr, B.ld)
    a, b = a.double(), b.double()
    if grad:
        Z, Y = ref.Buffer(z, pads[2], offsets[2]), ref.output(M, N, ot, pads[4], offsets[4])
        s = torch.full((N,), float("nan")).cuda() if sums else None
        fg.gemm16_grad(*common, ACT[act], Z.ptr, Z.ld, Y.ptr, Y.ld, s, ws, size, stream=stream)
        torch.cuda.synchronize()
        (y, dy), (cs, dcs) = ref.layer_grad(a, b, alpha, act, z.double())
        assert not ref.outside(Y.result(), y, dy, ot).any()
        if sums:
            assert not ref.outside(s.cpu(), cs, dcs, torch.float32).any()
        return Y.result(), s
    R = ref.Buffer(r, pads[3], offsets[3], ref.Buffer.SENTINEL if alias else float("nan"))
    Y = R if alias else ref.output(M, N, ot, pads[4], offsets[4])
    Z = ref.output(M, N, dt, pads[2], offsets[2]) if keep else None
    fg.gemm16(*common, bi.cuda() if bias else None, ACT[act], Z.ptr if keep else None, Z.ld if keep else 0, beta,
              R.ptr if beta else None, R.ld, Y.ptr, Y.ld, ws, size, stream=stream)
    torch.cuda.synchronize()
    (y, dy), (zw, dz) = ref.layer(a, b, alpha, bi.double() if bias else None, act, beta, r.double())
    if ints and not bias and act in ("none", "relu") and alpha == 1.0 and K < 1 << 20:
        dy, dz = 0 * dy, 0 * dz  # small integers: exact
    got = Y.result()
    bad = ref.outside(got, y, dy, ot)
    assert not bad.any(), "%d of %d wrong, first at %s: %s for %s" % (
        bad.sum(), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0], y[bad][0])
    if keep:
        assert not ref.outside(Z.result(), zw, dz, dt).any()
    return got, None


# Sizes where tiles, stages and the steps of the MMA end, and one past them.
SIZES = [(1, 1, 1), (1, 8, 8), (2, 3, 5), (16, 128, 64), (17, 129, 65), (31, 127, 63), (32, 256, 128), (33, 257, 129),
         (64, 100, 200), (128, 128, 1024), (129, 300, 77), (255, 383, 320), (257, 513, 100), (300, 70, 1030)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("ta,tb", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_integers_are_exact(M, N, K, ta, tb):
    product("bf16", M, N, K, out="f32", ta=ta, tb=tb, ints=True)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("act", ref.ACTS)
def test_layer(M, N, K, t, act):
    product(t, M, N, K, bias=True, act=act, keep=True, tb=M % 2)


@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("pads,offsets", [((0, 0, 0, 0, 0), (0, 0, 0, 0, 0)), ((1, 3, 1, 5, 3), (1, 1, 1, 1, 1)),
                                          ((8, 16, 2, 2, 2), (8, 0, 2, 2, 2)), ((0, 8, 1, 0, 4), (4, 8, 0, 3, 0)),
                                          ((7, 0, 0, 1, 2), (0, 2, 6, 0, 1))])
@pytest.mark.parametrize("M,N,K", [(50, 200, 72), (130, 131, 133), (1, 257, 129)])
def test_strides_and_alignment(t, out, pads, offsets, M, N, K):
    for ta, tb in ((0, 0), (1, 1)):
        product(t, M, N, K, out, ta, tb, 0.5, True, "silu", True, -0.5, pads=pads, offsets=offsets)
    product(t, M, N, K, out, grad=True, sums=True, act="gelu", pads=pads, offsets=offsets)


@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("M,N,K", [(40, 136, 96), (140, 99, 200)])
def test_added_to_what_is_there(t, out, M, N, K):
    product(t, M, N, K, out, beta=1.0, alias=True)
    product(t, M, N, K, out, beta=0.25, alpha=2.0, alias=True, bias=True, act="gelu", keep=True)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", ref.ACTS)
def test_gradient_through_an_activation(M, N, K, act):
    product("bf16", M, N, K, grad=True, sums=True, act=act, tb=True)
    product("f16", M, N, K, "f32", grad=True, sums=False, act=act, ta=True)


@pytest.mark.parametrize("alpha,K", [(0.0, 50), (1.0, 0), (0.0, 0)])
def test_no_products(alpha, K):
    """Neither operand is read: NaN in both."""
    M, N = 37, 141
    bias, r = torch.randn(N).cuda(), torch.randn(M, N).cuda()
    nan = torch.full((M * 64 + N * 64,), float("nan"), dtype=torch.bfloat16).cuda()
    y = torch.empty(M, N).cuda()
    fg.gemm16(fg.BF16, fg.F32, 0, 0, M, N, K, alpha, nan, max(K, 1), nan, N, bias, fg.ACT_RELU, None, 0, 2.0, r, N, y, N)
    want = bias.clamp(min=0) + 2 * r
    assert torch.equal(y, want)
    s = torch.full((N,), 5.0).cuda()
    ws = torch.empty(fg.gemm16_sums_workspace_size(1, M, N), dtype=torch.uint8).cuda()
    fg.gemm16_grad(fg.BF16, fg.F32, 0, 0, M, N, K, alpha, nan, max(K, 1), nan, N, fg.ACT_NONE, None, 0, y, N, s, ws, ws.numel())
    assert not y.any() and not s.any()


def test_not_finite():
    """NaN and infinities go where the formula takes them, and no further: rows and columns beside theirs are
    what they were.  beta == 0 does not read R; Z of -inf gives 0."""
    M, N, K = 40, 150, 70
    g = torch.Generator().manual_seed(3)
    a, b = torch.randn(M, K, generator=g).bfloat16(), torch.randn(K, N, generator=g).bfloat16()
    a[3, 5], a[20, 0], b[7, 100] = float("nan"), float("inf"), float("-inf")
    bias = torch.zeros(N)
    bias[9] = float("-inf")
    y = torch.empty(M, N, dtype=torch.bfloat16).cuda()
    z = torch.empty_like(y)
    nan = torch.full((M, N), float("nan"), dtype=torch.bfloat16).cuda()
    ws = torch.empty(fg.gemm16_copy_workspace_size(0, 0, 1, M, N, K), dtype=torch.uint8).cuda()
    for name in ref.ACTS:
        fg.gemm16(fg.BF16, fg.BF16, 0, 0, M, N, K, 1.0, a.cuda(), K, b.cuda(), N, bias.cuda(), ACT[name], z, N, 0.0, nan, N, y, N,
                  ws, ws.numel())
        (want, tol), (zw, _) = ref.layer(a.double(), b.double(), 1.0, bias.double(), name)
        tol = tol.nan_to_num(0, 0, 0)
        bad = ref.outside(y.cpu(), want, tol, torch.bfloat16)
        assert not bad.any(), (name, bad.nonzero()[:4], y.cpu()[bad][:4], want[bad][:4])
        assert torch.equal(z.cpu().isnan(), zw.isnan()) and torch.equal(z.cpu().isinf(), zw.isinf())
    # what is behind ReLU's gate does not matter
    gate = torch.randn(M, N, generator=g).bfloat16()
    gate[3], gate[20], gate[:, 100] = -1.0, 0.0, float("-inf")
    fg.gemm16_grad(fg.BF16, fg.BF16, 0, 0, M, N, K, 1.0, a.cuda(), K, b.cuda(), N, fg.ACT_RELU, gate.cuda(), N, y, N, None,
                   ws, ws.numel())
    assert y.isfinite().all() and not y[3].any() and not y[20].any() and not y[:, 100].any()


def test_slopes_at_the_ends():
    """act' of -inf, -30, 30, inf and NaN."""
    M, N = 3, 8
    z = torch.tensor([float("-inf"), -30.0, 0.0, 30.0, float("inf"), float("nan"), 1.0, -1.0]).repeat(M, 1).bfloat16()
    one = torch.ones(M, N, dtype=torch.bfloat16)
    d = torch.empty(M, N, dtype=torch.bfloat16).cuda()
    for name, zero in (("relu", 0.0), ("gelu", 0.5), ("silu", 0.5)):
        fg.act16_grad(fg.BF16, 1, M, N, None, ACT[name], one.cuda(), N, z.cuda(), N, d, N)
        got = d.cpu()[1]
        assert got[2:5].tolist() == [zero, 1.0, 1.0] and abs(got[0].item()) < 2e-7
        assert abs(got[1].item()) < 2e-7 and (got[5].isnan() or name == "relu")


@pytest.mark.parametrize("M,N,K", [(700, 1300, 520), (1111, 2050, 300), (2600, 700, 96), (520, 4100, 1000)])
@pytest.mark.parametrize("ta,tb", [(0, 0), (1, 1)])
def test_many_tiles(M, N, K, ta, tb):
    """Several tiles a CTA and tiles that end inside: exact."""
    product("f16", M, N, K, out="f32", ta=ta, tb=tb, ints=True, beta=1.0)
    product("bf16", M, N, K, ta=ta, tb=tb, grad=True, sums=True, act="relu")
