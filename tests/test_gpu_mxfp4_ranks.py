"""Products whose K is divided among the CTAs of a cluster: every number of CTAs that the plans give,
for tiles of 16, 32 and 64 rows, ragged in M, N and K, with exact sums.

Scales are 1/2, 1 and 2, so a partial sum is a multiple of 2^-4.  A product of random codes and scales has
a standard deviation of 15, a sum of 20001 of them one of 2100: far below 2^20, so that FP32 sums
are exact in any order."""

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


# a plan each of (16, 32, 64) rows and (1, 2, 4, 8) CTAs on 152 SMs, then the other ends of the ragged sizes
SHAPES = [(7, 200, 300), (1, 5000, 4101), (13, 201, 7000), (16, 100, 20001), (29, 300, 1030), (17, 5001, 4100), (30, 203, 7001),
          (29, 101, 20001), (60, 300, 300), (37, 5003, 4100), (63, 200, 7013), (60, 100, 20001), (130, 2100, 4100), (130, 1001, 11013)]


def test_the_shapes_reach_every_split():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plans = {divmod(fg.mxfp4_plan(fg.F32, *s, sms), 16) for s in SHAPES}
    assert plans == {(tile, ranks) for tile in (16, 32, 64) for ranks in (1, 2, 4, 8)}


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("t", TYPES)
def test_exact_sums(t, M, N, K):
    type_, dt = TYPES[t]
    rng = np.random.default_rng(M + N + K)
    (ca, sa), (cb, sb) = ref.random_codes(rng, M, K), ref.random_codes(rng, N, K)
    a, b = ref.values(ca, sa), ref.values(cb, sb)
    ld = 16 * ref.blocks(K) + 16
    ops = [torch.from_numpy(v).cuda() for v in (ref.pack_codes(ca, ld, 0x7D), ref.pack_scales(sa), ref.pack_codes(cb, ld, 0x7D),
                                                ref.pack_scales(sb))]
    bias = rng.integers(-40, 41, N) / 8.0
    c0 = torch.from_numpy(rng.integers(-8, 9, (M, N)) / 4.0).to(dt)
    out = torch.full((M, N + 3), -77.0, dtype=dt)
    out[:, :N] = c0
    out = out.cuda()
    fg.mxfp4_gemm(type_, M, N, K, 0.5, ops[0], ld, ops[1], ops[2], ld, ops[3], -2.0, out, N + 3,
                  torch.from_numpy(bias).float().cuda(), False)
    got = out.cpu()
    assert (got[:, N:] == -77.0).all()
    want = 0.5 * (a @ b.T) - 2.0 * c0.double().numpy() + bias
    assert np.abs(a @ b.T).max() < 2.0**16
    assert torch.equal(got[:, :N], torch.from_numpy(want).to(dt))
