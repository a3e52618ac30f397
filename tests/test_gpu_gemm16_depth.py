"""Sums of one sign over a long depth, where an accumulator that cuts falls short a little more with every addend.

Bounds, relative: half a step of the output, eps / 2; in turns of 768, at most a unit (2^-23) of the turn's sum for each of its 48
steps of 16 and as much again within a step: 96 * 2^-23 = 1.1e-5; and adding the turns up half a unit of the sum each:
K / 768 * 2^-24.  (In one go it would be K / 16 * 2^-23 and more: 7.8e-3 of a depth of 2^20.)"""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import gemm16_ref as ref
from test_gpu_gemm16 import CODE, _cuda  # noqa: F401

pytestmark = pytest.mark.gpu

TURNS = 16384


def positive(g, *shape, dtype):
    return torch.rand(*shape, generator=g, device="cuda").mul_(0.5).add_(0.5).to(dtype)


def summed(x, w):
    """x^T w in 64 bits, a part of the depth at a time."""
    return sum(a.double().t() @ b.double() for a, b in zip(x.split(1 << 16), w.split(1 << 16)))


def check(got, want, K, dtype, more=0.0):
    bound = torch.finfo(dtype).eps / 2 + 96 * 2.0**-23 + K / 768 * 2.0**-24 + more
    off = ((got.double() - want) / want).abs().max().item()
    assert off <= bound, "%g for %g" % (off, bound)


@pytest.mark.parametrize("t,K", [("f16", 1 << 18), ("f16", 1 << 20), ("bf16", 1 << 20), ("bf16", (1 << 20) + 77)])
@pytest.mark.parametrize("M,N", [(24, 128), (512, 2048)])
def test_products(t, K, M, N):
    dt = ref.TYPES[t]
    g = torch.Generator(device="cuda").manual_seed(0)
    x, w = positive(g, K, M, dtype=dt), positive(g, K, N, dtype=dt)
    alpha = 2.0**-10
    want = alpha * summed(x, w)
    assert fg.gemm16_plan(CODE[t], 0, 1, M, N, K, 0, 152) & TURNS
    # plain, and (a kernel of its own) with the sums kept and a residual
    y, z = torch.empty(M, N, dtype=dt, device="cuda"), torch.empty(M, N, dtype=dt, device="cuda")
    fg.gemm16(CODE[t], CODE[t], 1, 0, M, N, K, alpha, x, M, w, N, None, fg.ACT_RELU, None, 0, 0.0, None, 0, y, N)
    check(y, want, K, dt)
    r = positive(g, M, N, dtype=dt)
    fg.gemm16(CODE[t], CODE[t], 1, 0, M, N, K, alpha, x, M, w, N, None, fg.ACT_RELU, z, N, 64.0, r, N, y, N)
    check(z, want, K, dt)
    check(y, want + 64 * r.double(), K, dt, 2.0**-23)


@pytest.mark.parametrize("t", ["f16", "bf16"])
def test_weights_gradient_of_many_rows(t):
    dt, M, N, K, E = ref.TYPES[t], 1 << 20, 264, 136, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    x, d = positive(g, M, K, dtype=dt), positive(g, M, N, dtype=dt)
    at = [0, 1001, 1001, M]
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    c = torch.empty(E, K, N, dtype=dt, device="cuda")
    fg.gemm16_weight_grad(CODE[t], CODE[t], E, M, N, K, off, 2.0**-10, x, K, d, N, 0.0, c, N, K * N)
    assert not c[1].any()
    for e in (0, 2):
        i, j = at[e], at[e + 1]
        check(c[e], 2.0**-10 * summed(x[i:j], d[i:j]), j - i, dt)


@pytest.mark.parametrize("M,N", [(24, 128), (512, 2048)])
def test_gradients(M, N):
    """Through a gate, without column sums and with them."""
    K, dt = 1 << 18, torch.float16
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = positive(g, K, M, dtype=dt), positive(g, K, N, dtype=dt)
    want, z = 2.0**-10 * summed(x, w), torch.randn(M, N, generator=g, device="cuda").half()
    shut = z <= 0
    for s in (None, torch.empty(N, device="cuda")):
        y = torch.empty(M, N, dtype=dt, device="cuda")
        ws = torch.empty(fg.gemm16_sums_workspace_size(1, M, N), dtype=torch.uint8, device="cuda")
        fg.gemm16_grad(fg.F16, fg.F16, 1, 0, M, N, K, 2.0**-10, x, M, w, N, fg.ACT_RELU, z, N, y, N, s, ws, ws.numel())
        assert not y[shut].any()
        check(y[~shut], want[~shut], K, dt)
    sums = want.masked_fill(shut, 0).sum(0)  # M additions in FP32, each half a unit at most of a unit's magnitude
    open_ = sums > 0
    assert ((s.double() - sums).abs()[open_] <= (96 * 2.0**-23 + (K / 768 + M) * 2.0**-24) * sums[open_]).all()
