"""Scale bytes of rows beyond a matrix, which a product reads with their atom, may hold anything: its
outputs are those of zeros there."""

import numpy as np
import pytest
import torch

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    fg.library()
    fg.device_status(clear=True)
    yield
    assert fg.device_status() == fg.OK


def scales(s, fill):
    """Scale bytes packed, those of the rows beyond (and of the matrix's own blocks) being `fill`."""
    rows, nb = s.shape
    whole = np.full((-(-rows // 128) * 128, nb), fill, np.uint8)
    whole[:rows] = s
    return torch.from_numpy(ref.pack_scales(whole)).cuda()


# one plan of each kind, M and N in the middle of a group of 128 rows, even and odd numbers of blocks
@pytest.mark.parametrize("M,N,K", [(3, 140, 300), (3, 300, 4096), (20, 140, 320), (40, 200, 11008), (200, 140, 300), (1000, 2001, 300),
                                   (769, 9990, 2305), (2400, 1700, 4100)])
@pytest.mark.parametrize("fill", [255, 254])
def test_rows_beyond(M, N, K, fill):
    rng = np.random.default_rng(M + N)
    (ca, sa), (cb, sb) = ref.random_codes(rng, M, K), ref.random_codes(rng, N, K)
    ld = 16 * ref.blocks(K)
    a, b = torch.from_numpy(ref.pack_codes(ca)).cuda(), torch.from_numpy(ref.pack_codes(cb)).cuda()
    outs = []
    for f in (0, fill):
        out = torch.full((M, N), float("nan"), device="cuda")
        fg.mxfp4_gemm(fg.F32, M, N, K, 1.0, a, ld, scales(sa, f), b, ld, scales(sb, f), 0.0, out, N)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    assert torch.equal(outs[0].cpu(), torch.from_numpy(ref.values(ca, sa) @ ref.values(cb, sb).T).float())


@pytest.mark.parametrize("M", [1, 4, 9])
def test_rows_beyond_a_layers_weight(M):
    rng = np.random.default_rng(M)
    N, K = 200, 700
    code, s = ref.random_codes(rng, N, K)
    x = rng.integers(-4, 5, (M, K)).astype(float)
    out = torch.full((M, N), float("nan"), device="cuda")
    need = fg.mxfp4_linear_workspace_size(M, N, K)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    fg.mxfp4_linear(fg.F32, M, N, K, torch.from_numpy(x).float().cuda(), K, torch.from_numpy(ref.pack_codes(code)).cuda(),
                    16 * ref.blocks(K), scales(s, 255), None, False, out, N, ws, need)
    assert torch.equal(out.cpu(), torch.from_numpy(ref.through(x) @ ref.values(code, s).T).float())
