"""What the sources of the block-scaled kernels must not use."""
import glob
import os
import re

import pytest

import quantised_moe_expert_gb300 as qm

CSRC = os.path.join(os.path.dirname(qm.__file__), "csrc")
SOURCES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "scaled*.cu*")))


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_only_loads_beside_a_writing_predecessor(name):
    """These kernels start while their predecessor still writes what they read: the read-only path (ld.global.nc, by __ldg or
    const __restrict__) asks for memory that nobody writes while the kernel runs, and is not ordered by the wait for it."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.findall(r"__ldg\w*|ld\.global\.\S*nc|__restrict__|__restrict", code)


def test_the_family_is_found():
    assert {"scaled.cuh", "scaled_gemm.cu", "scaled_rows.cu", "scaled_vec.cu"} <= set(SOURCES)
