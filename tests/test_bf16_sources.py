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


def test_waits_that_run_out_are_met_by_all_threads_at_once():
    """In the norm's gradients a thread that gives up says so before a barrier and all read it behind that: a flag of the row's own, since
    a thread ahead may give up on the next row before the others have read this one's, and they would leave at different barriers.
    After the rows, what a thread met is its own."""
    with open(os.path.join(CSRC, "bf16_norm.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    code = code[code.index("gated_norm_grad_kernel("):code.index("gated_norm_sum_kernel(")]
    uses = re.findall(r"\bfailed\b(.{0,14})", code)
    assert len(uses) >= 4 and all(u.startswith("[") for u in uses), uses
    assert code.count("failed[which]") == 2 and "given_up(parity)" in code and "ph ^ 1, parity)" in code
