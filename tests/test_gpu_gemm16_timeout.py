"""Failure detection of the 16-bit products without a GPU fault, for every kind of kernel: a copy that never arrives.

The library's test hook makes a producer withhold one stage (of a pair's CTAs the first one's, so that the other
asks for copies that the first has not).  The bounded waits run out, the kernel records FGEMM_ERR_TIMEOUT,
waits for its copies and MMAs, frees its tensor memory and returns; the same context then computes the same call
as before."""

import time

import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
from test_gpu_gemm16 import _cuda  # noqa: F401

pytestmark = pytest.mark.gpu

LIMIT_NS = 200_000_000  # 0.2 s a wait
PAIR, TURNS = 8192, 16384
STAGE = 128  # the deepest


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def calls():
    """(name, plan, depth of a CTA, the call, its output)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    ws = torch.empty(1 << 23, dtype=torch.uint8, device="cuda")
    for M, N, K, tb in ((9, 304, 8200, 1), (40, 520, 4104, 0), (120, 1000, 1032, 1), (500, 2048, 1032, 0), (2500, 1000, 2056, 1),
                        (4100, 4104, 1032, 0)):
        a, b, r, z0 = randn(g, M, K), randn(g, N, K) if tb else randn(g, K, N), randn(g, M, N), randn(g, M, N)
        bias, z, y, s = torch.randn(N, generator=g, device="cuda"), torch.empty_like(r), torch.empty_like(r), torch.empty(N, device="cuda")
        ldb = K if tb else N
        shape = "%d x %d x %d" % (M, N, K)
        plan = fg.gemm16_plan(fg.BF16, 0, 1, M, N, K, 0, 152)
        yield "plain " + shape, plan, K, lambda M=M, N=N, K=K, tb=tb, a=a, b=b, ldb=ldb, y=y: fg.gemm16(
            fg.BF16, fg.BF16, 0, tb, M, N, K, 1.0, a, K, b, ldb, None, fg.ACT_NONE, None, 0, 0.0, None, 0, y, N), y
        yield "forward " + shape, plan, K, lambda M=M, N=N, K=K, tb=tb, a=a, b=b, ldb=ldb, y=y, z=z, r=r, bias=bias: fg.gemm16(
            fg.BF16, fg.BF16, 0, tb, M, N, K, 1.0, a, K, b, ldb, bias, fg.ACT_GELU, z, N, 1.0, r, N, y, N), y
        for sums, act in ((None, fg.ACT_GELU), (s, fg.ACT_SILU)):
            plan = fg.gemm16_plan(fg.BF16, 0, 1, M, N, K, sums is not None, 152)
            yield "gradient " + shape, plan, K, lambda M=M, N=N, K=K, tb=tb, a=a, b=b, ldb=ldb, y=y, z0=z0, sums=sums, act=act: fg.gemm16_grad(
                fg.BF16, fg.BF16, 0, tb, M, N, K, 1.0, a, K, b, ldb, act, z0, N, y, N, sums, ws, ws.numel()), y
    for rows, N, K in (([700, 650, 3, 1647], 1000, 776), ([3, 0, 150, 47], 136, 1032), ([2000, 2101], 2048, 2056)):
        E, M, at = len(rows), sum(rows), [0]
        for n in rows:
            at.append(at[-1] + n)
        off = torch.tensor(at, dtype=torch.int32, device="cuda")
        a, w, d, z0 = randn(g, M, K), randn(g, E, K, N), randn(g, M, N), randn(g, M, N)
        y, s, c = torch.empty_like(d), torch.empty(E, N, device="cuda"), torch.empty(E, K, N, device="cuda")
        plan = fg.gemm16_plan(fg.BF16, 1, E, M, N, K, 0, 152)
        yield "groups %s" % rows, plan, K, lambda M=M, N=N, K=K, E=E, off=off, a=a, w=w, y=y, d=d: fg.gemm16_grouped(
            fg.BF16, fg.BF16, 0, E, M, N, K, off, 1.0, a, K, w, N, K * N, None, fg.ACT_SILU, None, 0, 1.0, d, N, y, N), y
        plan = fg.gemm16_plan(fg.BF16, 1, E, M, N, K, 1, 152)
        yield "groups' gradient %s" % rows, plan, K, lambda M=M, N=N, K=K, E=E, off=off, a=a, w=w, y=y, z0=z0, s=s: fg.gemm16_grouped_grad(
            fg.BF16, fg.BF16, 0, E, M, N, K, off, 1.0, a, K, w, N, K * N, fg.ACT_GELU, z0, N, y, N, s, ws, ws.numel()), y
        plan = fg.gemm16_plan(fg.F32, 2, E, M, N, K, 0, 152)
        yield "weights %s" % rows, plan, max(rows), lambda M=M, N=N, K=K, E=E, off=off, a=a, d=d, c=c: fg.gemm16_weight_grad(
            fg.BF16, fg.F32, E, M, N, K, off, 1.0, a, K, d, N, 0.0, c, N, K * N), c


def test_kinds():
    plans = [plan for _, plan, *_ in calls()]
    assert {bool(p & PAIR) for p in plans} == {bool(p & TURNS) for p in plans} == {False, True}
    assert any(p % 16 > 1 for p in plans) and any(p & PAIR and p & TURNS for p in plans)


@pytest.mark.parametrize("withheld", [0, 1, 4])
def test_a_copy_that_never_arrives_is_reported(withheld):
    for name, plan, depth, call, out in calls():
        call()
        torch.cuda.synchronize()
        want = out.clone()
        assert fg.device_status(clear=True) == fg.OK
        try:
            fg.debug_withhold_tensor_core(withheld, LIMIT_NS)
            t0 = time.perf_counter()
            call()
            torch.cuda.synchronize()
            elapsed = time.perf_counter() - t0
        finally:
            fg.debug_withhold_tensor_core(-1)
        status = fg.device_status(clear=True)
        assert elapsed < 5.0, (name, elapsed)
        if depth // (plan % 16) > (withheld + 1) * STAGE:  # (a CTA has that many stages)
            assert status == fg.ERR_TIMEOUT, name
        out.fill_(float("nan"))
        call()
        torch.cuda.synchronize()
        assert fg.device_status() == fg.OK and torch.equal(out, want), name
