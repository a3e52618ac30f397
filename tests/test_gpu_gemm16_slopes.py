"""The activations' derivatives in the products' epilogue, at every 16-bit argument: the gradient of a product that is a
constant, in FP32, is the derivative as it is evaluated.

Bounds: gemm16_ref's, and for GELU left of -5.5, where Phi is taken as 0 and z as -5.5 before the bell:
Phi(z) + (|z| - 5.5) phi(z), and of 5.5 phi its own evaluation, (4 + 1.2 z^2) u.  The limits, 0 and 1, exactly."""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import gemm16_ref as ref
from test_gpu_gemm16 import ACT, CODE, _cuda  # noqa: F401

pytestmark = pytest.mark.gpu

PAIR, K = 8192, 8
TINY = 2.0**-120  # below it FP32's underflow counts


def arguments(dt):
    """Every value of the type, infinities and NaN among them, and some once more: a multiple of 16."""
    z = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
    return z[torch.randperm(65536, generator=torch.Generator().manual_seed(0))]


def bounds(z, name):
    want, tol = ref.slope(z, name)
    if name == "gelu":
        a = z.abs().clamp(max=50)
        left = ref.cdf(z) + (a - 5.5) * ref.phi(a) + (4 + 1.2 * a * a) * ref.U * 5.5 * ref.phi(a) + TINY
        want = torch.where(z == float("-inf"), 0.0, torch.where(z == float("inf"), 1.0, want))
        tol = torch.where(z < -5.5, left, tol)
    return want, torch.where(z.isinf(), 0.0, tol)


def check(got, z, name, scale):
    want, tol = bounds(z.double().cpu(), name)
    got = got.double().cpu() / scale
    nan = z.isnan().cpu()
    if name != "relu":  # (a closed gate)
        assert got[..., nan].isnan().all()
    off = (got - want).abs()[..., ~nan]
    assert (off <= tol[~nan]).all(), (name, z.cpu()[~nan][(off > tol[~nan]).any(0) if off.dim() > 1 else off > tol[~nan]][:8], off.max())


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("M,pad,sums", [(1, 0, False), (40, 0, False), (40, 1, False), (130, 8, True), (130, 2, True)])
def test_every_argument(t, name, M, pad, sums):
    """Single CTAs and pairs, Z through shared memory (rows on 16 bytes, pairs) and through registers."""
    dt = ref.TYPES[t]
    z = arguments(dt).cuda()
    N, scale = z.numel(), 4096.0
    assert bool(fg.gemm16_plan(fg.F32, 0, 1, M, N, K, sums, 152) & PAIR) == (M > 1)
    a, b = torch.zeros(M, K, dtype=dt, device="cuda"), torch.zeros(K, N, dtype=dt, device="cuda")
    a[:, 0], b[0] = 64.0, 64.0
    Z = torch.empty(M, N + pad, dtype=dt, device="cuda")
    Z[:, :N] = z
    y, s = torch.empty(M, N, device="cuda"), torch.empty(N, device="cuda") if sums else None
    ws = torch.empty(fg.gemm16_sums_workspace_size(1, M, N), dtype=torch.uint8, device="cuda")
    fg.gemm16_grad(CODE[t], fg.F32, 0, 0, M, N, K, 1.0, a, K, b, N, ACT[name], Z, N + pad, y, N, s, ws, ws.numel())
    assert all(torch.equal(y[0].nan_to_num(7), row.nan_to_num(7)) for row in y)
    check(y[0], z, name, scale)


@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
def test_limits_in_16_bits(name):
    """Gradients as large as F16 holds behind pre-activations that are closed."""
    M, N = 64, 512
    z = torch.tensor([float("-inf"), -60000.0, -100.0, -20.0]).repeat(N // 4).half().cuda().expand(M, N).contiguous()
    a, b = torch.zeros(M, K, dtype=torch.float16, device="cuda"), torch.zeros(K, N, dtype=torch.float16, device="cuda")
    a[:, 0], b[0] = 1.0, 60000.0
    y = torch.empty(M, N, dtype=torch.float16, device="cuda")
    off = torch.tensor([0, 20, M], dtype=torch.int32, device="cuda")
    fg.gemm16_grad(fg.F16, fg.F16, 0, 0, M, N, K, 1.0, a, K, b, N, ACT[name], z, N, y, N)
    # SiLU is s (1 + z (1 - s)), -20 sigma(-20) = -4e-8
    assert (y[:, :3] == 0).all() and (y.float().abs().max() < (0.003 if name == "silu" else 1e-7))
    y.fill_(9)
    fg.gemm16_grouped_grad(fg.F16, fg.F16, 0, 2, M, N, K, off, 1.0, a, K, b, N, 0, ACT[name], z, N, y, N)
    assert (y[:, :3] == 0).all()
