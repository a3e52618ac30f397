"""Failure detection of the MXFP4 products without a GPU fault: a copy that never arrives.

The library's test hook makes the producers withhold one stage.  The bounded waits run out after
a short limit, the kernel records FGEMM_ERR_TIMEOUT, drains its own copies and MMAs, frees its
tensor memory and returns, clusters and pairs included; the same context then computes the
same product exactly.
"""

import time

import numpy as np
import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

LIMIT_NS = 200_000_000  # 0.2 s a wait


@pytest.mark.parametrize("withheld", [0, 2])
@pytest.mark.parametrize("M,N,K,tile", [(3, 300, 4100, 0), (10, 130, 4100, 16), (40, 256, 11008, 64), (2600, 1400, 800, 128),
                                        (1700, 2900, 4100, 384), (2400, 1700, 4100, 512), (20, 300, 4100, -32)])
def test_withheld_stage_times_out_and_the_context_survives(M, N, K, tile, withheld):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if tile > 0:
        assert fg.mxfp4_plan(fg.F32, M, N, K, 152) // 16 == tile
    rng = np.random.default_rng(1)
    nb = ref.blocks(K)
    ca, sa = ref.random_codes(rng, M, K, 127, 128)
    cb, sb = ref.random_codes(rng, N, K, 127, 128)
    A, sA = torch.from_numpy(ref.pack_codes(ca)).cuda(), torch.from_numpy(ref.pack_scales(sa)).cuda()
    B, sB = torch.from_numpy(ref.pack_codes(cb)).cuda(), torch.from_numpy(ref.pack_scales(sb)).cuda()
    out = torch.empty(M, N, device="cuda")
    ws = torch.empty(max(16, fg.mxfp4_linear_workspace_size(M, N, K)), dtype=torch.uint8, device="cuda")
    x = torch.from_numpy(ref.values(ca, sa)).float().cuda()  # (whose quantised form has the same values)

    def call():
        if tile > 0:
            fg.mxfp4_gemm(fg.F32, M, N, K, 1.0, A, 16 * nb, sA, B, 16 * nb, sB, 0.0, out, N)
        else:  # tokens quantised in the product's kernel, and in a kernel before it
            fg.mxfp4_linear(fg.F32, M, N, K, x, K, B, 16 * nb, sB, None, False, out, N, ws, ws.numel())

    torch.cuda.synchronize()
    fg.device_status(clear=True)
    try:
        fg.debug_withhold_tensor_core(withheld, LIMIT_NS)
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        elapsed = time.perf_counter() - t0
    finally:
        fg.debug_withhold_tensor_core(-1)
    assert fg.device_status(clear=True) == fg.ERR_TIMEOUT
    assert elapsed < 5.0, "the bounded waits took %.2f s" % elapsed
    out.fill_(float("nan"))
    call()
    torch.cuda.synchronize()
    assert fg.device_status() == fg.OK
    want = torch.from_numpy(ref.values(ca, sa)).cuda() @ torch.from_numpy(ref.values(cb, sb)).cuda().t()
    assert torch.equal(out.double(), want)
