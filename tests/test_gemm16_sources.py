"""What the kernels of the 16-bit layers have to keep to, as the MXFP4 ones: each may be on the GPU while the
kernel before it still writes what it reads, so no loads through the non-coherent path."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_gemm_sm_gb300", "csrc")
FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "gemm16*.cu*")))


def test_there_are_sources():
    assert len(FILES) >= 8


@pytest.mark.parametrize("name", FILES)
def test_no_loads_through_the_non_coherent_path(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.findall(r"__ldg\b|__ldlu\b|ld\.global\.nc|ld\.nc|\btex\w*<|__restrict__", code)
