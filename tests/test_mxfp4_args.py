"""The MXFP4 entry points without a GPU: sizes, refusals before any launch, empty problems;
and the tests' own definition against values worked out by hand."""

import numpy as np
import pytest

import dense_fp32_gemm_sm_gb300 as fg
import mxfp4_ref as ref

FAKE = 0x10000  # a non-null, aligned address that validation never dereferences
INVALID, OK = fg.ERR_INVALID_VALUE, fg.OK


def test_sizes():
    assert fg.mxfp4_codes_size(1, 1) == 16
    assert fg.mxfp4_codes_size(7, 33) == 7 * 32
    assert fg.mxfp4_scales_size(1, 1) == 512
    assert fg.mxfp4_scales_size(128, 128) == 512
    assert fg.mxfp4_scales_size(129, 129) == 4 * 512
    assert fg.mxfp4_codes_size(0, 5) == 0 and fg.mxfp4_scales_size(5, -1) == 0
    assert fg.mxfp4_codes_size(2**31 - 256, 2**31 - 256) == (2**31 - 256) * 16 * (2**26 - 8)
    assert fg.mxfp4_quantize_grad_workspace_size(129, 10) == 2 * 10 * 4
    assert fg.mxfp4_quantize_grad_workspace_size(0, 10) == 0
    assert fg.mxfp4_linear_workspace_size(0, 5, 5) == 0
    assert fg.mxfp4_linear_workspace_size(4096, 4096, 4096) == 4096 * 2048 + 4096 * 128


def _quantize(**kw):
    a = dict(type=fg.F32, M=4, N=40, X=FAKE, ldx=40, row_codes=FAKE, ld_row_codes=32,
             row_scales=FAKE, col_codes=FAKE, ld_col_codes=16, col_scales=FAKE)
    a.update(kw)
    return fg.mxfp4_quantize(**a, check=False)


def _grad(**kw):
    a = dict(type=fg.BF16, M=4, N=40, G=FAKE, ldg=40, Y=FAKE, ldy=40, row_codes=FAKE,
             ld_row_codes=32, row_scales=FAKE, col_codes=FAKE, ld_col_codes=16, col_scales=FAKE,
             bias_grad=FAKE, workspace=FAKE, workspace_bytes=160)
    a.update(kw)
    return fg.mxfp4_quantize_grad(**a, check=False)


def _dequantize(**kw):
    a = dict(type=fg.F16, M=4, N=40, codes=FAKE, ld_codes=32, scales=FAKE, X=FAKE, ldx=40)
    a.update(kw)
    return fg.mxfp4_dequantize(**a, check=False)


def _gemm(**kw):
    a = dict(type=fg.F32, M=4, N=5, K=40, alpha=1.0, A_codes=FAKE, ld_A_codes=32, A_scales=FAKE,
             B_codes=FAKE, ld_B_codes=32, B_scales=FAKE, beta=0.0, C=FAKE, ldc=5, bias=FAKE)
    a.update(kw)
    return fg.mxfp4_gemm(**a, check=False)


def _linear(**kw):
    a = dict(type=fg.F32, M=300, N=5, K=40, X=FAKE, ldx=40, W_codes=FAKE, ld_W_codes=32,
             W_scales=FAKE, bias=None, apply_relu=False, Y=FAKE, ldy=5, workspace=FAKE,
             workspace_bytes=1 << 20)
    a.update(kw)
    return fg.mxfp4_linear(**a, check=False)


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(type=-1), dict(M=-1), dict(N=-1), dict(ldx=39), dict(X=None),
    dict(X=FAKE + 2), dict(type=fg.BF16, X=FAKE + 1), dict(row_codes=None), dict(row_scales=None),
    dict(col_codes=None), dict(col_scales=None), dict(ld_row_codes=16), dict(ld_row_codes=40),
    dict(ld_col_codes=0), dict(row_codes=FAKE + 8), dict(col_scales=FAKE + 4),
    dict(row_codes=None, row_scales=None, col_codes=None, col_scales=None),
])
def test_quantize_refuses(kw):
    assert _quantize(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(type=7), dict(M=-2), dict(ldg=39), dict(ldy=39), dict(G=None), dict(Y=FAKE + 1),
    dict(bias_grad=FAKE + 2), dict(workspace=None), dict(workspace=FAKE + 8),
    dict(workspace_bytes=159), dict(row_codes=None), dict(ld_row_codes=31),
])
def test_quantize_grad_refuses(kw):
    assert _grad(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(M=-1), dict(N=-1), dict(ldx=39), dict(X=None), dict(X=FAKE + 1),
    dict(codes=None), dict(scales=None), dict(ld_codes=16), dict(ld_codes=33),
    dict(codes=FAKE + 1), dict(scales=FAKE + 8),
])
def test_dequantize_refuses(kw):
    assert _dequantize(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(M=-1), dict(N=-1), dict(K=-1), dict(ld_A_codes=16), dict(ld_B_codes=16),
    dict(ld_A_codes=36), dict(A_codes=None), dict(A_scales=None), dict(B_codes=None),
    dict(B_scales=None), dict(A_codes=FAKE + 4), dict(B_scales=FAKE + 8), dict(C=None),
    dict(C=FAKE + 2), dict(ldc=4), dict(bias=FAKE + 1), dict(K=0, ld_A_codes=0),
])
def test_gemm_refuses(kw):
    assert _gemm(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(type=3), dict(M=-1), dict(K=-1), dict(ldx=39), dict(X=None), dict(X=FAKE + 2),
    dict(W_codes=None), dict(W_scales=None), dict(ld_W_codes=16), dict(Y=None), dict(ldy=4),
    dict(bias=FAKE + 2), dict(workspace=None), dict(workspace=FAKE + 4), dict(workspace_bytes=64),
])
def test_linear_refuses(kw):
    assert _linear(**kw) == INVALID


def test_empty_problems_do_nothing():
    assert _quantize(M=0) == OK and _quantize(N=0, X=None) == OK
    assert _grad(N=0) == OK and _grad(M=0, bias_grad=None) == OK
    assert _dequantize(M=0, X=None) == OK and _dequantize(N=0) == OK
    assert _gemm(M=0) == OK and _gemm(N=0, C=None) == OK
    assert _linear(M=0, workspace=None) == OK and _linear(N=0) == OK


def test_sizes_beyond_the_limit_are_not_supported():
    big = 2**31 - 255
    assert _quantize(M=big, ld_col_codes=2**30) == fg.ERR_NOT_SUPPORTED
    assert _dequantize(M=big) == fg.ERR_NOT_SUPPORTED
    assert _gemm(M=big) == fg.ERR_NOT_SUPPORTED


def test_binding_checks_tensor_types():
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError):
        _quantize(X=torch.zeros(4, 40))
    with pytest.raises(TypeError):
        _gemm(A_codes=torch.zeros(4, 32, dtype=torch.uint8))


def test_plan():
    plan = lambda *a: divmod(fg.mxfp4_plan(*a), 16)  # noqa: E731
    # few rows: narrow tiles, a long K over a few tiles divided, one or two B tiles an SM not
    assert plan(fg.F32, 1, 11008, 4096, 152) == (16, 1)
    assert plan(fg.F32, 20, 4096, 11008, 152) == (32, 4)
    assert plan(fg.F32, 130, 1001, 11013, 152) == (64, 4)
    assert plan(fg.F32, 256, 256, 256, 152) == (64, 1)
    # a rank never goes without stages of 256
    for K in (1, 256, 257, 600, 1025):
        for M in (1, 17, 33):
            assert 1 <= plan(fg.BF16, M, 128, K, 152)[1] <= -(-K // 256)
    # large products: pairs of CTAs, in the tile that wastes less of the last round
    assert plan(fg.BF16, 8192, 11008, 4096, 152) in ((384, 0), (512, 0))
    assert plan(fg.BF16, 2048, 4096, 11008, 152) == (512, 0)
    assert plan(fg.F32, 8000, 1000, 4000, 152) == (512, 0)
    assert plan(fg.F32, 4096, 4096, 1024, 152) == (128, 0)
    for bad in ((3, 4, 4, 4, 152), (0, 0, 4, 4, 152), (0, 4, 4, 0, 152), (0, 4, 4, 4, 1), (0, 2**31 - 1, 4, 4, 152)):
        assert fg.mxfp4_plan(*bad) == -1


def test_definition_by_hand():
    # largest 7: floor(log2 7) = 2, scale 2^0; 7 saturates to 6; ties go to the even code
    x = [7.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.26, -0.0]
    code, s = ref.encode(np.array([x]))
    assert s.tolist() == [[127]]
    assert code[0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 14, 1, 8]
    # the smallest scale: 2^-127 for a block of subnormals, and for a block of zeros
    code, s = ref.encode(np.array([[2.0**-127, 2.0**-149, 0.0]]))
    assert s.tolist() == [[0]] and code[0].tolist() == [2, 0, 0]
    code, s = ref.encode(np.zeros((1, 33)))
    assert s.tolist() == [[0, 0]] and not code.any()
    # a NaN spoils its block and no other
    x = np.ones((1, 64))
    x[0, 3] = np.inf
    code, s = ref.encode(x)
    assert s.tolist() == [[255, 125]] and code[0, :32].max() == 0 and code[0, 32] == 6
    v = ref.values(code, s)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_calls_convert_what_they_are_given():
    # NULL for None and 0, a truth value for the ReLU, floats or whole numbers for alpha and beta
    assert _gemm(M=0, alpha=1, beta=0, bias=0, apply_relu=1) == OK
    assert _gemm(A_codes=0) == INVALID
    assert _quantize(M=0, stream=1) == OK
    for wrong in (dict(M=2**40), dict(ldx="40"), dict(M=1.5)):
        with pytest.raises((TypeError, OverflowError)):
            _quantize(**wrong)
    with pytest.raises(TypeError):
        _quantize(X=object())
    with pytest.raises(TypeError):
        _gemm(alpha="1")
    with pytest.raises((TypeError, OverflowError)):
        _linear(workspace_bytes=-1)
    with pytest.raises(fg.FgemmError) as e:
        fg.mxfp4_dequantize(fg.F32, -1, 5, FAKE, 16, FAKE, FAKE, 5)
    assert e.value.status == INVALID
