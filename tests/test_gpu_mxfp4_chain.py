"""A call's output as the next call's tokens or bias, with nothing in between.

A product that adds to its C (beta) brings old values of C near the SMs, and the kernel after it
is there before it ends: what that one reads has to be what was written all the same.  The
results have to equal those of the same calls with a wait after each."""

import numpy as np
import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": (fg.F32, torch.float32), "bf16": (fg.BF16, torch.bfloat16), "f16": (fg.F16, torch.float16)}
ROUNDS = 12


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    fg.library()
    fg.device_status(clear=True)
    yield
    assert fg.device_status() == fg.OK


def matrix(rng, rows, cols, lo=118, hi=122):
    code, s = ref.random_codes(rng, rows, cols, lo, hi)
    return torch.from_numpy(ref.pack_codes(code)).cuda(), 16 * ref.blocks(cols), torch.from_numpy(ref.pack_scales(s)).cuda()


def both_ways(run):
    """run(after each call) with a wait and without one: the same bits."""
    one, row = run(torch.cuda.synchronize), run(lambda: None)
    torch.cuda.synchronize()
    assert len(one) == len(row) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(one, row))
    assert all(torch.isfinite(a).all() for a in one)
    assert len({tuple(a.flatten()[:64].tolist()) for a in one}) == len(one), "every round gives other values"


@pytest.mark.parametrize("M,K,N", [(1, 512, 1000), (1, 4096, 300), (4, 1000, 2000), (4, 4096, 513), (30, 700, 400), (200, 512, 300)])
@pytest.mark.parametrize("t", TYPES)
def test_an_output_as_the_next_calls_tokens(t, M, K, N):
    type_, dt = TYPES[t]
    rng = np.random.default_rng(M + K + N)
    A, B, W = matrix(rng, M, 96), matrix(rng, K, 96), matrix(rng, N, K)
    start = torch.from_numpy(rng.standard_normal((M, K))).to(dt).cuda()
    need = fg.mxfp4_linear_workspace_size(M, N, K)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def run(after):
        c, outs = start.clone(), torch.full((ROUNDS, M, N), float("nan"), dtype=dt, device="cuda")
        torch.cuda.synchronize()
        for y in outs:
            fg.mxfp4_gemm(type_, M, K, 96, 1.0, *A, *B, -0.9375, c, K)
            after()
            fg.mxfp4_linear(type_, M, N, K, c, K, *W, None, False, y, N, ws, need)
            after()
        return list(outs)

    both_ways(run)


# one product for each kernel: 16, 32 and 64 rows, with a long K divided, 128 x 128, pairs
@pytest.mark.parametrize("M,N,K", [(3, 1000, 512), (3, 300, 4096), (20, 700, 300), (60, 500, 6000), (1000, 2000, 300),
                                   (2400, 1700, 4100)])
def test_an_output_as_the_next_calls_bias(M, N, K):
    rng = np.random.default_rng(M + N + K)
    A, B = matrix(rng, M, K), matrix(rng, N, K)
    a, b = matrix(rng, 1, 96), matrix(rng, N, 96)
    start = torch.from_numpy(rng.standard_normal((1, N))).float().cuda()
    rounds = ROUNDS if M < 1000 else 4

    def run(after):
        bias, outs = start.clone(), torch.full((rounds, M, N), float("nan"), device="cuda")
        torch.cuda.synchronize()
        for y in outs:
            fg.mxfp4_gemm(fg.F32, 1, N, 96, 1.0, *a, *b, -0.9375, bias, N)
            after()
            fg.mxfp4_gemm(fg.F32, M, N, K, 1.0, *A, *B, 0.0, y, N, bias, False)
            after()
        return list(outs)

    both_ways(run)


@pytest.mark.parametrize("M", [1, 4])
def test_an_output_as_the_bias_of_the_next_tokens(M):
    rng = np.random.default_rng(M)
    N, K = 1500, 1024
    W, a, b = matrix(rng, N, K), matrix(rng, 1, 96), matrix(rng, N, 96)
    x = torch.from_numpy(rng.standard_normal((M, K))).float().cuda()
    start = torch.from_numpy(rng.standard_normal((1, N))).float().cuda()

    def run(after):
        bias, outs = start.clone(), torch.full((ROUNDS, M, N), float("nan"), device="cuda")
        torch.cuda.synchronize()
        for y in outs:
            fg.mxfp4_gemm(fg.F32, 1, N, 96, 1.0, *a, *b, -0.9375, bias, N)
            after()
            fg.mxfp4_linear(fg.F32, M, N, K, x, K, *W, bias, False, y, N)
            after()
        return list(outs)

    both_ways(run)
