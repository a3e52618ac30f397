"""A NaN under ReLU: a spoiled block's elements stand for NaN, so the outputs that they reach are NaN
with the activation as without it, whichever kernel runs the product."""

import numpy as np
import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": (fg.F32, torch.float32), "bf16": (fg.BF16, torch.bfloat16), "f16": (fg.F16, torch.float16)}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    fg.library()
    fg.device_status(clear=True)
    yield
    assert fg.device_status() == fg.OK


def spoiled(rng, rows, cols, row):
    """Codes, leading dimension and scales on the GPU, and the values: the last block of a row is NaN."""
    code, s = ref.random_codes(rng, rows, cols)
    s[row, -1] = 255
    code[row, 32 * (s.shape[1] - 1):] = 0
    return (torch.from_numpy(ref.pack_codes(code)).cuda(), 16 * ref.blocks(cols), torch.from_numpy(ref.pack_scales(s)).cuda()), ref.values(code, s)


def check(got, want, dt):
    """want: exact in FP32 (sums of small multiples of 2^-4)."""
    want = torch.from_numpy(want).to(dt)
    got = got.cpu()
    assert torch.equal(got.isnan(), want.isnan()) and want.isnan().any() and not want.isnan().all()
    assert torch.equal(got.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))


def relu(x):
    return np.where(np.isnan(x), x, np.maximum(x, 0))


# a plan of each kind: 16, 32 and 64 rows, K divided or not, 128 x 128, pairs of 192 and of 256 rows
SHAPES = [(3, 140, 300), (3, 300, 4096), (20, 140, 300), (40, 200, 11008), (200, 140, 300), (1000, 2000, 300), (2400, 1700, 4100),
          (769, 9990, 2305)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("t", TYPES)
def test_products(t, M, N, K):
    type_, dt = TYPES[t]
    rng = np.random.default_rng(K)
    (A, a), (B, b) = spoiled(rng, M, K, 1), spoiled(rng, N, K, N - 2)
    out = torch.empty(M, N, dtype=dt, device="cuda")
    scale = 2.0**-6 if t == "f16" else 1.0  # (a power of two; keeps f16 in its range)
    fg.mxfp4_gemm(type_, M, N, K, scale, *A, *B, 0.0, out, N, None, True)
    check(out, scale * relu(a @ b.T), dt)
    # a NaN in C or in the bias
    c = torch.zeros(M, N, dtype=dt, device="cuda")
    c[-1, 0] = float("nan")
    bias = torch.zeros(N, device="cuda")
    bias[2] = float("nan")
    fg.mxfp4_gemm(type_, M, N, K, scale, *A, *B, 1.0, c, N, bias, True)
    want = scale * relu(a @ b.T)
    want[-1, 0] = want[:, 2] = np.nan
    check(c, want, dt)


def test_the_shapes_reach_every_kernel():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = {fg.mxfp4_plan(fg.F32, *s, sms) // 16 for s in SHAPES}
    assert tiles == {16, 32, 64, 128, 384, 512}


@pytest.mark.parametrize("t", TYPES)
def test_no_products(t):
    type_, dt = TYPES[t]
    c = torch.tensor([[-1.0, 2.0, float("nan")], [3.0, -4.0, 5.0]], dtype=dt, device="cuda")
    bias = torch.tensor([float("nan"), 1.0, 1.0], device="cuda")
    fg.mxfp4_gemm(type_, 2, 3, 0, 1.0, None, 16, None, None, 16, None, 1.0, c, 3, bias, True)
    n = float("nan")
    assert torch.equal(c.cpu().float().nan_to_num(nan=-1.0), torch.tensor([[n, 3.0, n], [n, 0.0, 6.0]]).nan_to_num(nan=-1.0))


@pytest.mark.parametrize("M,N,K", [(1, 200, 300), (2, 300, 4096), (4, 1001, 700), (9, 300, 700), (70, 300, 700)])
@pytest.mark.parametrize("t", TYPES)
def test_the_layer_on_a_spoiled_token(t, M, N, K):
    type_, dt = TYPES[t]
    rng = np.random.default_rng(N)
    W, w = spoiled(rng, N, K, N - 2)
    x = rng.integers(-4, 5, (M, K)).astype(float)  # (whole numbers that quantising leaves alone)
    if M > 1:
        x[1, 40] = np.inf
    X = torch.from_numpy(x).to(dt).cuda()
    out = torch.empty(M, N, dtype=dt, device="cuda")
    need = fg.mxfp4_linear_workspace_size(M, N, K)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    fg.mxfp4_linear(type_, M, N, K, X, K, *W, None, True, out, N, ws, need)
    q = ref.through(x)
    check(out, relu(q @ w.T), dt)
    for i in range(M):  # and one that is spoiled as a whole
        assert out[i].isnan().all() == (M > 1 and i == 1)
