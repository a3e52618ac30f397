"""What the MXFP4 kernels' sources have to keep to.

Every MXFP4 kernel may be on the GPU while the kernel before it still writes what it reads.
Loads through the non-coherent path (ld.global.nc, __ldg) want memory that nobody writes
while the kernel runs, so none may be there: a stale value is a race that no run has to show."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_gemm_sm_gb300", "csrc")
FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "mxfp4*.cu*")))


@pytest.mark.parametrize("name", FILES)
def test_no_loads_through_the_non_coherent_path(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.findall(r"__ldg\b|__ldlu\b|ld\.global\.nc|ld\.nc|\btex\w*<|__restrict__", code)
