"""Which depths of the 16-bit products are added up in turns, on the CPU."""

import pytest

import dense_fp32_gemm_sm_gb300 as fg

TURNS = 16384


@pytest.mark.parametrize("out,sums,most", [(fg.F32, 0, 768), (fg.BF16, 1, 768), (fg.F16, 1, 768), (fg.F16, 0, 1 << 14), (fg.BF16, 0, 1 << 17)])
@pytest.mark.parametrize("M,N", [(1, 8), (300, 200), (4096, 4096)])
def test_plans(out, sums, most, M, N):
    for grouped in (0, 1):
        assert not fg.gemm16_plan(out, grouped, 1, M, N, most, sums, 152) & TURNS
        assert fg.gemm16_plan(out, grouped, 1, M, N, most + 1, sums, 152) & TURNS
    if not sums:  # all groups' rows count: one of them may have them all
        assert not fg.gemm16_plan(out, 2, 5, most, N, M, 0, 152) & TURNS
        assert fg.gemm16_plan(out, 2, 5, most + 1, N, M, 0, 152) & TURNS
