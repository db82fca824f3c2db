"""The build checks what a kernel's launch depends on and the compiler decides."""
import os

import pytest

from gaussian_splatting_differentiable_gs_gb300 import build

LOG = """ptxas info    : Compiling entry function '_ZN2gs12wgrad_kernelIfEEvv' for 'sm_103a'
ptxas info    : Function properties for _ZN2gs12wgrad_kernelIfEEvv
    8 bytes stack frame, 12 bytes spill stores, 32 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers, 8 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN2gs17wgrad_join_kernelIfEEvv' for 'sm_103a'
ptxas info    : Function properties for _ZN2gs17wgrad_join_kernelIfEEvv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 32 registers, used 0 barriers
"""


def test_registers_that_a_launch_shares_out_are_checked():
    """Roles of the weight gradient's kernel share out the registers of its launch: with
    any other number than the source states, each call would be refused at run time."""
    src = os.path.join(build.CSRC, "wgrad.cu")
    build._check_registers(src, LOG % 96)
    for log in (LOG % 88, LOG % 104, "", LOG.replace("Used %d registers", "Used no registers")):
        with pytest.raises(RuntimeError, match="registers"):
            build._check_registers(src, log)
    build._check_registers(os.path.join(build.CSRC, "rope.cu"), "")  # nothing to check there
