"""The 16-bit entry points without a GPU: sizes, refusals before any launch, empty problems, plans."""

import pytest

import dense_fp32_gemm_sm_gb300 as fg

FAKE = 0x10000  # a non-null, aligned address that validation never dereferences
INVALID, OK, UNSUPPORTED = fg.ERR_INVALID_VALUE, fg.OK, fg.ERR_NOT_SUPPORTED
BIG = 2**31 - 1


def _gemm(**kw):
    a = dict(type=fg.BF16, out_type=fg.BF16, transa=0, transb=0, M=4, N=5, K=40, alpha=1.0, A=FAKE, lda=40, B=FAKE, ldb=8, bias=FAKE,
             act=fg.ACT_GELU, Z=FAKE, ldz=5, beta=1.0, R=FAKE, ldr=5, Y=FAKE, ldy=5)
    a.update(kw)
    return fg.gemm16(**a, check=False)


def _grad(**kw):
    a = dict(type=fg.F16, out_type=fg.F32, transa=0, transb=1, M=4, N=5, K=40, alpha=1.0, A=FAKE, lda=40, B=FAKE, ldb=40,
             act=fg.ACT_SILU, Z=FAKE, ldz=5, Y=FAKE, ldy=5, col_sums=FAKE, workspace=FAKE, workspace_bytes=1 << 20)
    a.update(kw)
    return fg.gemm16_grad(**a, check=False)


def _grouped(**kw):
    a = dict(type=fg.BF16, out_type=fg.F32, transb=0, groups=3, M=4, N=8, K=40, offsets=FAKE, alpha=1.0, A=FAKE, lda=40, B=FAKE,
             ldb=8, strideB=320, bias=FAKE, act=fg.ACT_RELU, Z=FAKE, ldz=8, beta=0.5, R=FAKE, ldr=8, Y=FAKE, ldy=8)
    a.update(kw)
    return fg.gemm16_grouped(**a, check=False)


def _grouped_grad(**kw):
    a = dict(type=fg.BF16, out_type=fg.BF16, transb=1, groups=3, M=4, N=8, K=40, offsets=FAKE, alpha=1.0, A=FAKE, lda=40, B=FAKE,
             ldb=40, strideB=320, act=fg.ACT_RELU, Z=FAKE, ldz=8, Y=FAKE, ldy=8, col_sums=FAKE, workspace=FAKE,
             workspace_bytes=1 << 20)
    a.update(kw)
    return fg.gemm16_grouped_grad(**a, check=False)


def _weight_grad(**kw):
    a = dict(type=fg.BF16, out_type=fg.F32, groups=3, M=4, N=8, K=40, offsets=FAKE, alpha=1.0, A=FAKE, lda=40, G=FAKE, ldg=8, beta=1.0,
             C=FAKE, ldc=8, strideC=320)
    a.update(kw)
    return fg.gemm16_weight_grad(**a, check=False)


def _act(**kw):
    a = dict(type=fg.F16, groups=3, M=4, N=8, offsets=FAKE, act=fg.ACT_GELU, G=FAKE, ldg=8, Z=FAKE, ldz=8, D=FAKE, ldd=8,
             col_sums=FAKE, workspace=FAKE, workspace_bytes=1 << 20)
    a.update(kw)
    return fg.act16_grad(**a, check=False)


def test_sizes():
    assert fg.gemm16_copy_workspace_size(0, 0, 1, 3, 5, 7) == 256 + 7 * 8 * 2  # A 3 x 8, B 7 x 8
    assert fg.gemm16_copy_workspace_size(1, 1, 2, 3, 5, 7) == 256 + 2 * 5 * 8 * 2  # A 7 x 8, B 5 x 8 twice
    assert fg.gemm16_copy_workspace_size(0, 0, 0, 3, 5, 7) == fg.gemm16_copy_workspace_size(0, 2, 1, 3, 5, 7) == 0
    assert fg.gemm16_copy_workspace_size(0, 0, 1, 0, 5, 7) == 0
    # two rows of partial sums for every 32 rows and for every group, and where each group's start
    assert fg.gemm16_sums_workspace_size(1, 33, 10) == 256 + 256
    assert fg.gemm16_sums_workspace_size(5, 64, 100) == -(-2 * 7 * 100 * 4 // 256) * 256 + 256
    assert fg.gemm16_sums_workspace_size(1, 0, 10) == 0
    assert fg.gemm16_copy_workspace_size(0, 0, 1000, BIG, BIG, BIG) > 2**63  # saturates, never wraps


@pytest.mark.parametrize("kw", [
    dict(type=fg.F32), dict(type=3), dict(out_type=fg.F16), dict(out_type=4), dict(transa=2), dict(transb=-1), dict(M=-1), dict(N=-1),
    dict(K=-1), dict(lda=39), dict(ldb=4), dict(transa=1, lda=3), dict(transb=1), dict(A=None), dict(B=None), dict(A=FAKE + 1),
    dict(B=FAKE + 1), dict(bias=FAKE + 2), dict(act=4), dict(act=-1), dict(Z=FAKE + 1), dict(ldz=4), dict(ldr=4), dict(R=None),
    dict(R=FAKE + 1), dict(out_type=fg.F32, R=FAKE + 2), dict(out_type=fg.F32, Y=FAKE + 2), dict(Y=None), dict(ldy=4),
    dict(A=FAKE + 2),               # a copy is wanted: no workspace
    dict(ldb=9), dict(lda=41, workspace=FAKE, workspace_bytes=4 * 80 - 1),
    dict(lda=41, workspace=FAKE + 8, workspace_bytes=1 << 20),
])
def test_gemm_refuses(kw):
    assert _gemm(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(act=9), dict(Z=None), dict(Z=FAKE + 1), dict(ldz=4), dict(Y=None), dict(ldy=4), dict(col_sums=FAKE + 2),
                                dict(workspace=None), dict(workspace_bytes=263), dict(workspace=FAKE + 4), dict(out_type=fg.BF16)])
def test_grad_refuses(kw):
    assert _grad(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(groups=0), dict(groups=-1), dict(offsets=None), dict(offsets=FAKE + 2), dict(strideB=-8),
                                dict(strideB=321), dict(transb=7), dict(K=48), dict(Y=None), dict(R=None), dict(Z=FAKE + 1)])
def test_grouped_refuses(kw):
    assert _grouped(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(groups=0), dict(offsets=None), dict(Z=None), dict(workspace=None), dict(workspace_bytes=271),
                                dict(ldb=39), dict(col_sums=FAKE + 1)])
def test_grouped_grad_refuses(kw):
    assert _grouped_grad(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(groups=0), dict(offsets=None), dict(strideC=319), dict(strideC=-1), dict(ldc=7), dict(lda=39),
                                dict(ldg=7), dict(C=None), dict(C=FAKE + 2), dict(A=None), dict(G=None), dict(ldg=9), dict(type=fg.F32),
                                dict(out_type=fg.F16), dict(M=-1)])
def test_weight_grad_refuses(kw):
    assert _weight_grad(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(type=fg.F32), dict(groups=0), dict(offsets=None), dict(act=5), dict(G=None), dict(Z=None), dict(ldg=7),
                                dict(ldz=7), dict(ldd=7), dict(D=FAKE + 1), dict(D=None, col_sums=None), dict(col_sums=FAKE + 2),
                                dict(workspace=None), dict(workspace_bytes=100), dict(workspace=FAKE + 2), dict(N=-1)])
def test_act_grad_refuses(kw):
    assert _act(**kw) == INVALID


def test_sizes_beyond_the_limits_are_not_supported():
    assert _gemm(M=BIG) == UNSUPPORTED
    assert _grouped(groups=fg.MAX_GROUPS + 1) == _weight_grad(groups=fg.MAX_GROUPS + 1) == _act(groups=fg.MAX_GROUPS + 1) == UNSUPPORTED
    assert _act(M=BIG, workspace_bytes=1 << 62) == UNSUPPORTED


def test_empty_problems():
    assert _gemm(M=0, A=None, Y=None) == _gemm(N=0, B=None, Y=None, ldb=1) == OK
    assert _grouped(M=0, A=None, Y=None, offsets=None) == _weight_grad(K=0, A=None, C=None) == _weight_grad(N=0, C=None) == OK
    assert _act(N=0, G=None) == OK
    assert _grad(N=0, col_sums=None, Y=None) == OK


def test_plans():
    """Every kind of plan is chosen for some sizes, and what a plan promises holds."""
    plan = lambda *a: fg.gemm16_plan(*a, 152)  # noqa: E731
    kinds = set()
    for M in (1, 5, 16, 33, 77, 128, 200, 333, 512, 1000, 2048, 4100, 8192):
        for N in (1, 100, 256, 1001, 2048, 4096, 11008):
            for K in (1, 64, 500, 1237, 4096, 11008):
                for sums in (0, 1):
                    v = plan(fg.BF16, 0, 1, M, N, K, sums)
                    pair, rows, ranks, turns = bool(v & 8192), (v & 8191) // 16, v % 16, bool(v & 16384)
                    kinds.add((pair, rows, ranks > 1))
                    assert rows in ((64, 96, 128, 160, 192, 224, 256) if pair else (16, 32, 64)) and 1 <= ranks <= 8
                    assert not (sums and (ranks > 1 or rows < 32)) and (ranks == 1 or not pair)
                    assert turns == (bool(sums) and K > 768)
    assert len(kinds) >= 10
    assert plan(fg.F32, 0, 1, 100, 100, 769, 0) & 16384 and not plan(fg.F32, 0, 1, 100, 100, 768, 0) & 16384
    for bad in ((fg.BF16, 3, 1, 4, 4, 4, 0), (fg.BF16, 1, 0, 4, 4, 4, 0), (fg.BF16, 1, 1025, 4, 4, 4, 0), (fg.BF16, 0, 1, 0, 4, 4, 0),
                (fg.BF16, 0, 1, 4, 4, BIG, 0)):
        assert plan(*bad) == -1
    assert fg.gemm16_plan(fg.BF16, 0, 1, 4, 4, 4, 0, 1) == -1


@pytest.mark.parametrize("M", [1, 31, 32, 33, 63, 64, 100, 1000, 8192, 100000])
@pytest.mark.parametrize("groups", [1, 2, 7, 64, 1024])
@pytest.mark.parametrize("N", [1, 300, 5000])
def test_partial_sums_fit_their_room(M, groups, N):
    """The room of fgemm_gemm16_sums_workspace_size against the rows of partial sums that are written: two for each
    tile of rows, of which each group with rows may have one that is not full."""
    room = fg.gemm16_sums_workspace_size(groups, M, N)
    rows = (fg.gemm16_plan(fg.BF16, 1, groups, M, N, 512, 1, 152) & 8191) // 16
    worst = M // rows + min(groups, M)
    assert 2 * worst * N * 4 <= room
