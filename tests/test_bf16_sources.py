"""What the sources of the 16-bit kernels must not use."""
import glob
import os
import re

import pytest

import quantised_moe_expert_gb300 as qm

CSRC = os.path.join(os.path.dirname(qm.__file__), "csrc")
SOURCES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "bf16*.cu*")) + [os.path.join(CSRC, "f32x2.cuh")])


@pytest.mark.parametrize("name", SOURCES)
def test_no_read_only_loads_beside_a_writing_predecessor(name):
    """These kernels start while their predecessor still writes what they read (see test_scaled_sources.py)."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.findall(r"__ldg\w*|ld\.global\.\S*nc|__restrict__|__restrict", code)


@pytest.mark.parametrize("name", [n for n in SOURCES if n.endswith(".cu") and n != "bf16_api.cu"])
def test_every_kernel_waits_for_its_predecessor(name):
    with open(os.path.join(CSRC, name)) as f:
        code = f.read()
    kernels = code.count("__global__ void")
    assert kernels and len(re.findall(r"\bpdl_wait\(\);", code)) == kernels == len(re.findall(r"\bpdl_trigger\(\);", code))
