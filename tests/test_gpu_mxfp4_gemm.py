"""Products of MXFP4 matrices on the GPU against the definition in 64 bits.

Tolerances.  A product of two codes times its power-of-two scales is exact, and so is the
sum over a block (a multiple of 1/4 of its scales below 2^11).  What rounds is the sum over
the nb = ceil(K/32) blocks in FP32 (each addition by at most one unit in the last place,
2^-23, of a partial sum that is at most mag = sum |a||b|), alpha, beta * C and the bias, all
in FP32: the value before the rounding to C's type lies within
    tol = ((nb + 3) * |alpha| mag + 2 |beta C0| + |bias|) * 2^-23 + 2^-24 |C_ref|
of C_ref.  Rounding to nearest is monotone, so C lies between C_ref - tol and C_ref + tol,
both rounded to its type.  Where all partial sums are small multiples of one power of two,
FP32 results are exact and equal.
"""

import numpy as np
import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": (fg.F32, torch.float32), "bf16": (fg.BF16, torch.bfloat16), "f16": (fg.F16, torch.float16)}
SENTINEL = -77.0


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    fg.library()
    fg.device_status(clear=True)
    yield
    assert fg.device_status() == fg.OK


def operand(rng, rows, K, lo=126, hi=129, extra=0):
    code, s = ref.random_codes(rng, rows, K, lo, hi)
    # bytes between the rows hold codes that must not count
    codes = torch.from_numpy(ref.pack_codes(code, 16 * ref.blocks(K) + extra, 0x7D)).cuda()
    return codes, codes.shape[1], torch.from_numpy(ref.pack_scales(s)).cuda(), ref.values(code, s)


def outside(got, want, tol, dt):
    """Which elements are not between want - tol and want + tol, rounded to the type."""
    to = lambda x: torch.from_numpy(x).to(dt).double().numpy()  # noqa: E731
    return ~((got >= to(want - tol)) & (got <= to(want + tol)))


def product(t, M, N, K, alpha=1.0, beta=0.0, bias=False, relu=False, lo=126, hi=129, extra=(0, 0), pad=0, offset=0,
            seed=0, c_nan=False, stream=None):
    code, dt = TYPES[t]
    rng = np.random.default_rng(seed)
    A, B = operand(rng, M, K, lo, hi, extra[0]), operand(rng, N, K, lo, hi, extra[1])
    ld = N + pad
    c0 = torch.from_numpy(rng.integers(-8, 9, (M, N)) / 4.0).to(dt)
    buf = torch.full((M * ld + offset + 8,), SENTINEL, dtype=dt)
    view = buf[offset:offset + M * ld].view(M, ld)
    view[:, :N] = float("nan") if c_nan else c0
    out = buf.cuda()
    b = torch.from_numpy(rng.integers(-40, 41, N) / 8.0).float().cuda() if bias else None
    fg.mxfp4_gemm(code, M, N, K, alpha, A[0], A[1], A[2], B[0], B[1], B[2], beta,
                  out.data_ptr() + offset * out.element_size(), ld, b, relu, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    got = out.cpu()
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside[offset:offset + M * ld].view(M, ld)[:, :N] = True
    assert (got[~inside] == SENTINEL).all(), "written outside C"
    got = got[offset:offset + M * ld].view(M, ld)[:, :N].double().numpy()
    want = alpha * (A[3] @ B[3].T)
    mag = abs(alpha) * (np.abs(A[3]) @ np.abs(B[3]).T)
    tol = (ref.blocks(K) + 3) * mag
    if beta:
        want = want + beta * c0.double().numpy()
        tol = tol + 2 * np.abs(beta * c0.double().numpy())
    if bias:
        want = want + b.double().cpu().numpy()
        tol = tol + np.abs(b.double().cpu().numpy())
    if relu:
        want = np.maximum(want, 0)
    tol = tol * 2.0**-23 + 2.0**-24 * np.abs(want)
    return got, want, tol, dt


def check(*a, **kw):
    got, want, tol, dt = product(*a, **kw)
    bad = outside(got, want, tol, dt)
    assert not bad.any(), "%d of %d outside, first at %s: %r, not %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0])


def check_exact(*a, **kw):
    got, want, _, dt = product(*a, **kw)
    want = torch.from_numpy(want).float().to(dt).double().numpy()
    bad = got != want
    assert not bad.any(), "%d of %d differ, first at %s: %r, not %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0])


# M from one row to several tiles of any height, N around the 128 rows of an MMA, K below and
# beyond one block, one 64-deep MMA, one 256-deep stage
SHAPES = [(1, 1, 1), (1, 1000, 4096), (2, 128, 32), (5, 130, 64), (8, 128, 40), (9, 257, 256), (16, 100, 96), (17, 384, 257),
          (31, 640, 1030), (32, 128, 512), (33, 129, 320), (63, 127, 2048), (64, 256, 768), (65, 1000, 100),
          (127, 128, 129), (128, 128, 128), (129, 130, 1000), (255, 500, 544), (256, 256, 256), (257, 300, 33),
          (300, 2000, 700), (1000, 1001, 999), (2600, 1400, 320)]
# Products that run by pairs of CTAs: one round and several, ragged in every size.
PAIRS = [(2400, 1700, 4100), (1700, 2900, 4100), (5000, 5001, 2100), (769, 9990, 2305)]


def test_the_shapes_reach_every_kernel():
    tiles = {fg.mxfp4_plan(fg.F32, *s, 152) // 16 for s in SHAPES + PAIRS}
    assert tiles == {16, 32, 64, 128, 384, 512}
    ranks = {fg.mxfp4_plan(fg.F32, *s, 152) % 16 for s in SHAPES + [(130, 300, 40001), (40, 200, 11008)]}
    assert ranks >= {0, 1, 4}


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_sums(M, N, K):
    # scales 1/2, 1, 2: every partial sum is a multiple of 2^-4 below 2^20, exact in FP32
    check_exact("f32", M, N, K, seed=M + N + K)


@pytest.mark.parametrize("M,N,K", PAIRS)
def test_exact_sums_by_pairs(M, N, K):
    # (K * 144 < 2^20: as above)
    check_exact("f32", M, N, K, bias=True, pad=1, seed=M + N + K)


@pytest.mark.parametrize("M,N,K", SHAPES[::3] + PAIRS[:1])
@pytest.mark.parametrize("t", TYPES)
def test_epilogue(t, M, N, K):
    check(t, M, N, K, alpha=1.5 * 2.0**-7, beta=-0.75, bias=True, relu=True, pad=3, offset=1, seed=1)
    check(t, M, N, K, alpha=-2.0**-8, bias=True, pad=8, seed=2, c_nan=True)


@pytest.mark.parametrize("M,N,K", SHAPES[1::4] + PAIRS[:1])
@pytest.mark.parametrize("t", TYPES)
def test_scales_of_many_sizes(t, M, N, K):
    # scales over 2^-12 .. 2^11; padded rows of codes
    check(t, M, N, K, alpha=2.0**-9 if t == "f16" else 1.0, lo=115 if t != "f16" else 122, hi=139 if t != "f16" else 130,
          extra=(16, 48), seed=3)


def test_long_sum():
    check("f32", 130, 300, 40001, lo=120, hi=132, seed=4)
    check_exact("f32", 40, 200, 11008, seed=5)


def test_products_at_the_ends_of_the_range():
    # scales 2^-126 * 2^126: the product's scale is formed without passing through either end
    rng = np.random.default_rng(6)
    K = 256
    ca, sa = ref.random_codes(rng, 40, K, 1, 2)
    cb, sb = ref.random_codes(rng, 130, K, 253, 254)
    out = torch.empty(40, 130, device="cuda")
    fg.mxfp4_gemm(fg.F32, 40, 130, K, 1.0, torch.from_numpy(ref.pack_codes(ca)).cuda(), 128,
                  torch.from_numpy(ref.pack_scales(sa)).cuda(), torch.from_numpy(ref.pack_codes(cb)).cuda(), 128,
                  torch.from_numpy(ref.pack_scales(sb)).cuda(), 0.0, out, 130)
    want = ref.values(ca, sa) @ ref.values(cb, sb).T
    assert np.array_equal(out.cpu().numpy(), want)


@pytest.mark.parametrize("M,N,K", [(3, 140, 300), (200, 140, 300), (300, 500, 1000)])
def test_nan_blocks_spoil_their_rows_and_columns_alone(M, N, K):
    rng = np.random.default_rng(7)
    ca, sa = ref.random_codes(rng, M, K)
    cb, sb = ref.random_codes(rng, N, K)
    sa[1, -1] = 255
    sb[139, 0] = 255
    ca[1, -1 - (K - 1) % 32:] = 0  # as quantising leaves such a block
    cb[139, :32] = 0
    out = torch.empty(M, N, device="cuda")
    nb = ref.blocks(K)
    fg.mxfp4_gemm(fg.F32, M, N, K, 1.0, torch.from_numpy(ref.pack_codes(ca)).cuda(), 16 * nb,
                  torch.from_numpy(ref.pack_scales(sa)).cuda(), torch.from_numpy(ref.pack_codes(cb)).cuda(), 16 * nb,
                  torch.from_numpy(ref.pack_scales(sb)).cuda(), 0.0, out, N)
    want = ref.values(ca, sa) @ ref.values(cb, sb).T
    got = out.cpu().numpy()
    assert np.isnan(want[1]).all() and np.isnan(want[:, 139]).all()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


@pytest.mark.parametrize("t", TYPES)
def test_no_products(t):
    code, dt = TYPES[t]
    c0 = torch.arange(-20, 19, dtype=torch.float32).view(3, 13).to(dt)
    bias = torch.arange(13, dtype=torch.float32, device="cuda") - 6
    for kw in (dict(K=0, alpha=1.0), dict(K=64, alpha=0.0)):
        c = c0.cuda()
        fg.mxfp4_gemm(code, 3, 13, kw["K"], kw["alpha"], None, 32, None, None, 32, None, 0.5, c, 13, bias, True)
        want = (0.5 * c0.float() + bias.cpu()).clamp(min=0).to(dt)
        assert torch.equal(c.cpu(), want)
        c.fill_(float("nan"))
        fg.mxfp4_gemm(code, 3, 13, kw["K"], kw["alpha"], None, 32, None, None, 32, None, 0.0, c, 13)
        assert not c.any()


def test_same_result_every_time():
    outs = [product("f32", 200, 300, 5000, lo=115, hi=139, seed=8)[0] for _ in range(3)]
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


# ---- the layer on unquantised tokens ----------------------------------------------------


def linear(t, M, N, K, bias=True, relu=False, pad=0, offset=0, seed=0, x=None):
    code, dt = TYPES[t]
    rng = np.random.default_rng(seed)
    if x is None:
        x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-3, 3, (M, 1)))
        x[rng.random((M, K)) < 0.01] *= 16
    ldx = K + pad
    xb = torch.full((M * ldx + offset + 8,), float("nan"), dtype=dt)
    xv = xb[offset:offset + M * ldx].view(M, ldx)
    xv[:, :K] = torch.from_numpy(x).to(dt)
    xd = xb.cuda()
    W = operand(rng, N, K, 120, 124, extra=16)
    b = torch.from_numpy(rng.standard_normal(N)).float().cuda() if bias else None
    out = torch.full((M, N + pad), SENTINEL, dtype=dt, device="cuda")
    need = fg.mxfp4_linear_workspace_size(M, N, K)
    ws = torch.full((max(need, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    fg.mxfp4_linear(code, M, N, K, xd.data_ptr() + offset * xd.element_size(), ldx, W[0], W[1], W[2], b, relu, out, N + pad,
                    ws if need else None, need)
    torch.cuda.synchronize()
    assert (out[:, N:] == SENTINEL).all()
    q = ref.through(xv[:, :K].double().numpy())
    want = q @ W[3].T
    tol = (ref.blocks(K) + 3) * (np.abs(q) @ np.abs(W[3]).T)
    if bias:
        want = want + b.double().cpu().numpy()
        tol = tol + np.abs(b.double().cpu().numpy())
    if relu:
        want = np.maximum(want, 0)
    got = out[:, :N].double().cpu().numpy()
    tol = tol * 2.0**-23 + 2.0**-24 * np.abs(want)
    return got, want, tol, dt


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 32, 33, 64, 65, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (127, 33), (130, 64), (1001, 1237), (256, 4096), (700, 4100)])
def test_linear(M, N, K):
    assert not outside(*linear("f32", M, N, K, relu=M % 2 == 0, pad=M % 3, offset=M % 2, seed=M * N + K)).any()


@pytest.mark.parametrize("M", [1, 4, 6, 20, 140])
@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,pad", [(300, 999, 1), (1024, 2048, 0), (64, 11008, 8)])
def test_linear_types(t, M, N, K, pad):
    assert not outside(*linear(t, M, N, K, bias=M != 4, pad=pad, seed=9)).any()


@pytest.mark.parametrize("M,K", [(1, 30000), (4, 43008), (4, 43009), (2, 60001)])
def test_linear_long_sums(M, K):
    # quantised tokens of up to 168 stages of 256 fit in a cluster's shared memory
    assert (fg.mxfp4_linear_workspace_size(M, 200, K) == 0) == (K <= 43008)
    assert not outside(*linear("f32", M, 200, K, seed=K)).any()


@pytest.mark.parametrize("M", [1, 3, 40, 200])
def test_linear_without_anything_to_sum(M):
    y = torch.full((M, 9), float("nan"), device="cuda")
    bias = torch.arange(9, dtype=torch.float32, device="cuda") - 4
    fg.mxfp4_linear(fg.F32, M, 9, 0, None, 1, None, 16, None, bias, True, y, 9)
    assert torch.equal(y, bias.clamp(min=0).expand(M, 9))


@pytest.mark.parametrize("M", [2, 50])
def test_linear_with_a_token_of_nan(M):
    x = np.ones((M, 200))
    x[1, 40] = np.nan
    got, want, tol, _ = linear("f32", M, 70, 200, x=x)
    assert np.isnan(got[1]).all() and np.isnan(want[1]).all()
    assert (np.abs(got[0] - want[0]) <= tol[0]).all()


# ---- a layer's training step ------------------------------------------------------------


def quantised(x, t=fg.F32):
    M, N = x.shape
    mk = lambda r, c: (torch.empty(r, 16 * ref.blocks(c), dtype=torch.uint8, device="cuda"),  # noqa: E731
                       torch.empty(fg.mxfp4_scales_size(r, c), dtype=torch.uint8, device="cuda"))
    r, c = mk(M, N), mk(N, M)
    fg.mxfp4_quantize(t, M, N, x, N, r[0], r[0].shape[1], r[1], c[0], c[0].shape[1], c[1])
    return r, c


def test_backward_is_the_gradient_of_the_layer():
    # Values that quantising leaves alone (E2M1 values, one scale), so that the layer is the
    # exact Y = ReLU(X W + b) and its differences are exact: the loss sum(Y * G) against
    # steps of one element, both ways.
    rng = np.random.default_rng(11)
    M, N, K = 70, 45, 40
    # every block holds a 4 (scale 2^0), whichever way it runs
    draw = lambda r, c: np.where(rng.random((r, c)) < 0.5, 4.0, rng.choice([0.0, 1, 2, 3, -1, -2, -4], (r, c)))  # noqa: E731
    X, W, G = draw(M, K), draw(K, N), draw(M, N)
    for m in (X, W, G):
        assert np.array_equal(ref.through(m), m) and np.array_equal(ref.through(m.T).T, m)
    pre = X @ W - 50.5
    Y = np.maximum(pre, 0)
    gate = lambda m: np.where(Y > 0, m, 0)  # noqa: E731
    assert np.array_equal(ref.through(gate(G)), gate(G)) and np.array_equal(ref.through(gate(G).T).T, gate(G))
    dev = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    (xr, xc), (wr, wc) = quantised(dev(X)), quantised(dev(W))
    y = torch.empty(M, N, device="cuda")
    b = torch.full((N,), -50.5, device="cuda")
    fg.mxfp4_gemm(fg.F32, M, N, K, 1.0, xr[0], xr[0].shape[1], xr[1], wc[0], wc[0].shape[1], wc[1], 0.0, y, N, b, True)
    assert np.array_equal(y.cpu().numpy(), Y)
    ld = lambda c: 16 * ref.blocks(c)  # noqa: E731
    mk = lambda r, c: (torch.empty(r, ld(c), dtype=torch.uint8, device="cuda"),  # noqa: E731
                       torch.empty(fg.mxfp4_scales_size(r, c), dtype=torch.uint8, device="cuda"))
    gr, gc = mk(M, N), mk(N, M)
    db, ws = torch.empty(N, device="cuda"), torch.empty(4 * N, dtype=torch.uint8, device="cuda")
    g = dev(G)
    fg.mxfp4_quantize_grad(fg.F32, M, N, g, N, y, N, gr[0], ld(N), gr[1], gc[0], ld(M), gc[1], db, ws, ws.numel())
    dx, dw = torch.empty(M, K, device="cuda"), torch.empty(K, N, device="cuda")
    fg.mxfp4_gemm(fg.F32, M, K, N, 1.0, gr[0], ld(N), gr[1], wr[0], ld(N), wr[1], 0.0, dx, K)
    fg.mxfp4_gemm(fg.F32, K, N, M, 1.0, xc[0], ld(M), xc[1], gc[0], ld(M), gc[1], 0.0, dw, N)
    assert np.array_equal(dx.cpu().numpy(), gate(G) @ W.T)
    assert np.array_equal(dw.cpu().numpy(), X.T @ gate(G))
    assert np.array_equal(db.cpu().numpy(), gate(G).sum(0))
    loss = lambda X, W, b: (np.maximum(X @ W + b, 0) * G).sum()  # noqa: E731
    h = 2.0**-6  # no pre-activation (a whole number + 1/2) changes sign for steps of h * 4
    for _ in range(40):
        i, k, j = rng.integers(M), rng.integers(K), rng.integers(N)
        d = np.zeros((M, K))
        d[i, k] = h
        assert (loss(X + d, W, -50.5) - loss(X - d, W, -50.5)) / (2 * h) == dx[i, k].item()
        d = np.zeros((K, N))
        d[k, j] = h
        assert (loss(X, W + d, -50.5) - loss(X, W - d, -50.5)) / (2 * h) == dw[k, j].item()


def test_offsets_beyond_32_bits():
    # C with more than 2^31 elements, rows of codes at byte offsets beyond 2^31
    M, N, K = 70001, 32771, 64
    rng = np.random.default_rng(12)
    ca, sa = ref.random_codes(rng, 11, K)
    cb, sb = ref.random_codes(rng, 13, K)
    ia, ib = torch.arange(M) % 11, torch.arange(N) % 13
    ld = 32768  # a long pitch: A's last row starts beyond 2^31 bytes
    A = torch.full((M, ld), 0x7D, dtype=torch.uint8, device="cuda")
    A[:, :32] = torch.from_numpy(ref.pack_codes(ca))[ia].cuda()
    sA = torch.from_numpy(ref.pack_scales(sa[ia.numpy()])).cuda()
    B = torch.from_numpy(ref.pack_codes(cb))[ib].cuda()
    sB = torch.from_numpy(ref.pack_scales(sb[ib.numpy()])).cuda()
    C = torch.empty(M, N, device="cuda")
    fg.mxfp4_gemm(fg.F32, M, N, K, 1.0, A, ld, sA, B, 32, sB, 0.0, C, N)
    torch.cuda.synchronize()
    want = torch.from_numpy((ref.values(ca, sa) @ ref.values(cb, sb).T)).float().cuda()
    for i in range(0, M, 8192):
        ii = ia[i:i + 8192].cuda()
        assert torch.equal(C[i:i + 8192], want[ii][:, ib.cuda()])
