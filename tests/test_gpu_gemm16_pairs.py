"""GELU, SiLU and ReLU in the kernels of CTA pairs, forward and gradient, plain and by groups, in both types, against 64 bits.

Operands are integers and sixteenths whose products and sums FP32 holds, so that all that may be off is the
activation's own evaluation (bounds: gemm16_ref), a rounding where R comes in, one a row in column sums, and the output's."""

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import gemm16_ref as ref
from test_gpu_gemm16 import ACT, CODE, _cuda  # noqa: F401

pytestmark = pytest.mark.gpu

PAIR, TURNS = 8192, 16384
# M, N, K: tiles of 96 to 256 rows, depths to either side of a turn; columns by 8 and not.
SHAPES = [(1100, 1304, 200), (1500, 1304, 776), (2500, 1000, 136), (900, 2904, 1032), (5000, 2601, 72), (4100, 4104, 1608), (1801, 1290, 264)]
ROWS = [700, 0, 3, 1500, 260, 31, 606]  # of seven groups, and 17 rows of none behind them


def operands(g, t, out, M, N, K, E=None):
    dt = ref.TYPES[t]
    lead = () if E is None else (E,)
    a = torch.randint(-1, 2, (M, K), generator=g, device="cuda").to(dt)
    b = (torch.randint(-3, 4, (*lead, K, N), generator=g, device="cuda") / 16.0).to(dt)
    bias = torch.randint(-8, 9, (*lead, N), generator=g, device="cuda") / 4.0
    r = torch.randn(M, N, generator=g, device="cuda").to(ref.TYPES[out])
    z = 2 * torch.randn(M, N, generator=g, device="cuda")
    z[::7, ::5], z[1::7, 1::5], z[2::7, 3::5] = float("-inf"), float("inf"), -9.5
    return a, b, bias, r, z.to(dt)


def room(*sizes):
    ws = torch.full((sum(sizes),), 255, dtype=torch.uint8, device="cuda")
    return ws, ws.numel()


def padded(M, N, dtype, pad, fill):
    return torch.full((M, N + pad), fill, dtype=dtype, device="cuda")


def inside(got, want, tol, dtype, what):
    bad = ref.outside(got, want, tol, dtype)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[bad][0].item())


def check_forward(y, z, p, bias, r, beta, name, dt, ot):
    p = p + bias.double()
    want, tol = ref.act(p, name)
    tol = tol + ref.U * ((beta * r.double()).abs() + want.abs() + tol)
    inside(y, want + beta * r.double(), tol, ot, "Y")
    assert torch.equal(z, p.to(dt))


def check_gradient(y, s, p, z, name, ot):
    slope, ds = ref.slope(z.double(), name)
    want, tol = p * slope, p.abs() * ds + ref.U * (p * slope).abs()
    inside(y, want, tol, ot, "dZ")
    if s is not None:
        total = tol.sum(0) + (y.shape[0] + 1) * ref.U * (want.abs() + tol).sum(0)
        inside(s, want.sum(0), total, torch.float32, "sums")


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_forward(M, N, K, t, out, name):
    dt, ot = ref.TYPES[t], ref.TYPES[out]
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a, b, bias, r, _ = operands(g, t, out, M, N, K)
    assert fg.gemm16_plan(CODE[out], 0, 1, M, N, K, 0, 152) & PAIR
    p = a.double() @ b.double()
    for pad in (0, 1):
        y, z = padded(M, N, ot, pad, 7.0), padded(M, N, dt, pad, 7.0)
        fg.gemm16(CODE[t], CODE[out], 0, 0, M, N, K, 1.0, a, K, b, N, bias, ACT[name], z, N + pad, -0.5, r, N, y, N + pad,
                  *room(fg.gemm16_copy_workspace_size(0, 0, 1, M, N, K)))
        check_forward(y[:, :N], z[:, :N], p, bias, r, -0.5, name, dt, ot)
        assert (y[:, N:] == 7).all() and (z[:, N:] == 7).all()


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("name", ["relu", "gelu", "silu"])
def test_gradient(M, N, K, t, out, name):
    """Z by rows on 16 bytes (through shared memory where it has room) and not, with column sums and without."""
    dt, ot = ref.TYPES[t], ref.TYPES[out]
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a, b, _, _, z0 = operands(g, t, out, M, N, K)
    p = a.double() @ b.double()
    for sums in (False, True):
        plan = fg.gemm16_plan(CODE[out], 0, 1, M, N, K, sums, 152)
        assert plan & PAIR and bool(plan & TURNS) == (K > 768 and (sums or out == "f32"))
        for pad in (0, 2, 8):
            z, y = padded(M, N, dt, pad, float("nan")), padded(M, N, ot, pad, 7.0)
            z[:, :N] = z0
            s = torch.full((N,), float("nan"), device="cuda") if sums else None
            fg.gemm16_grad(CODE[t], CODE[out], 0, 0, M, N, K, 1.0, a, K, b, N, ACT[name], z, N + pad, y, N + pad, s,
                           *room(fg.gemm16_copy_workspace_size(0, 0, 1, M, N, K), fg.gemm16_sums_workspace_size(1, M, N)))
            check_gradient(y[:, :N], s, p, z0, name, ot)
            assert (y[:, N:] == 7).all()


@pytest.mark.parametrize("N,K", [(2904, 264), (2904, 1032), (2899, 200)])
@pytest.mark.parametrize("t,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("name", ["gelu", "silu"])
def test_groups(N, K, t, out, name):
    dt, ot = ref.TYPES[t], ref.TYPES[out]
    E, used = len(ROWS), sum(ROWS)
    M = used + 17
    at = [0]
    for n in ROWS:
        at.append(at[-1] + n)
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(N + K)
    a, b, bias, r, z0 = operands(g, t, out, M, N, K, E)
    for sums in (False, True):
        assert fg.gemm16_plan(CODE[out], 1, E, M, N, K, sums, 152) & PAIR
    copies = fg.gemm16_copy_workspace_size(0, 0, E, M, N, K)
    y, z = padded(M, N, ot, 0, 7.0), padded(M, N, dt, 0, 7.0)
    fg.gemm16_grouped(CODE[t], CODE[out], 0, E, M, N, K, off, 1.0, a, K, b, N, K * N, bias, ACT[name], z, N, 2.0, r, N, y, N,
                      *room(copies))
    d, s = padded(M, N, ot, 0, 7.0), torch.full((E, N), float("nan"), device="cuda")
    fg.gemm16_grouped_grad(CODE[t], CODE[out], 0, E, M, N, K, off, 1.0, a, K, b, N, K * N, ACT[name], z0, N, d, N, s,
                           *room(copies, fg.gemm16_sums_workspace_size(E, M, N)))
    d2 = padded(M, N, ot, 0, 7.0)
    fg.gemm16_grouped_grad(CODE[t], CODE[out], 0, E, M, N, K, off, 1.0, a, K, b, N, K * N, ACT[name], z0, N, d2, N, None, *room(copies))
    assert torch.equal(d, d2)  # (exact sums: in turns or in one go)
    for e, (i, j) in enumerate(zip(at, at[1:])):
        p = a[i:j].double() @ b[e].double()
        check_forward(y[i:j], z[i:j], p, bias[e], r[i:j], 2.0, name, dt, ot)
        check_gradient(d[i:j], s[e], p, z0[i:j], name, ot)
    for rest in (y, z, d):
        assert (rest[used:] == 7).all()
