"""The build's check of the kernels whose warps share out the launch's registers."""
import re

import pytest

from chunked_gated_delta_bwd_gb300 import build

LINE = """ptxas info    : Compiling entry function '%s' for 'sm_103a'
ptxas info    : Function properties for %s
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 16 barriers, 16 bytes smem
"""
WALK, OTHER = "_ZN3gdr12_GLOBAL__N_15k_dlaILi128ELi3EEEvNS0_5WalksIXT0_EEENS0_4GridE", "_ZN3gdr12_GLOBAL__N_110k_dla_tailILi64ELi1EEEvv"
WIDE, NARROW = "_ZN3gdr12_GLOBAL__N_18k_linearILb1ELi256EEEvv", "_ZN3gdr12_GLOBAL__N_18k_linearILb1ELi128EEEvv"


def log(*kernels):
    return "".join(LINE % (name, name, regs) for name, regs in kernels)


def test_registers_checked():
    build.check_registers("gdr_dla.cu", log((OTHER, 162), (WALK, 96), (OTHER, 40)))
    build.check_registers("gdr_linear.cu", log((NARROW, 166), (WIDE, 168)))
    build.check_registers("gdr_norm.cu", log((WALK, 12)))
    for src, bad in (("gdr_dla.cu", log((OTHER, 96), (WALK, 95))), ("gdr_linear.cu", log((WIDE, 170), (NARROW, 168)))):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_registers(src, bad)


def test_registers_are_those_of_the_kernels():
    """The numbers beside the kernels, and that each name is found there."""
    read = lambda name: open(build.os.path.join(build.CSRC, name)).read()  # noqa: E731
    assert int(re.search(r"REGS = (\d+),", read("gdr_dla.cu")).group(1)) == build.REGISTERS["gdr_dla.cu"][1]
    assert int(re.search(r"regs != (\d+)\)", read("gdr_linear.cu")).group(1)) == build.REGISTERS["gdr_linear.cu"][1]
