"""What a call needs to have been built."""

import sysconfig

import pytest

import dense_fp32_gemm_sm_gb300 as fg
from dense_fp32_gemm_sm_gb300 import _binding, _build


def no_compiler(*a, **kw):
    raise RuntimeError("no Python headers")


def test_the_library_does_without_the_python_module(monkeypatch):
    # FP32 calls go through ctypes: neither a C compiler nor Python's headers are wanted for them
    monkeypatch.setattr(_build, "build_calls", no_compiler)
    monkeypatch.setattr(_binding, "_lib", None)
    monkeypatch.setattr(_binding, "_calls", None)
    assert fg.select_config(0, 0, 64, 64, 64, 1, True, 152) >= 0
    assert fg.mxfp4_codes_size(1, 1) == 16
    with pytest.raises(RuntimeError, match="headers"):
        fg.mxfp4_dequantize(fg.F32, 0, 0, None, 16, None, None, 1)


def test_the_python_module_belongs_to_its_interpreter():
    assert _build.CALLS.endswith("_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
    assert _build.build_calls() == _build.CALLS == _binding._native().__file__
