"""The build's check of the 8-bit head's tile kernels (CPU only): planted
registers in accumulators and scratch are found, MFMAs are not."""

import os

import pytest

from rollout_logprob_consistency_amd import isa_check

CLEAN = """
_ZN2lp11tile_kernelE:
	v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], 0
	v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]
	v_accvgpr_read_b32 v8, a0
.Lfunc_end0:
_ZN2lp13stream_kernelE:
	v_accvgpr_write_b32 a0, v1
.Lfunc_end1:
"""


def test_clean_kernels_pass():
    assert isa_check.check_no_parked_registers(CLEAN, "tile_kernel") == []


@pytest.mark.parametrize("line", ["v_accvgpr_write_b32 a0, v218", "scratch_store_dword off, v0, off",
                                  "scratch_load_dwordx2 v[0:1], off, off offset:12"])
def test_planted_ones_are_found(line):
    planted = CLEAN.replace("\tv_accvgpr_read_b32 v8, a0", "\t%s\n\tv_accvgpr_read_b32 v8, a0" % line)
    problems = isa_check.check_no_parked_registers(planted, "tile_kernel")
    assert len(problems) == 1 and "tile_kernel" in problems[0]


def test_a_missing_kernel_is_a_problem():
    assert isa_check.check_no_parked_registers(CLEAN, "no_such_kernel")


def test_the_built_kernels():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "_build",
                        "int8.device.s")
    if not os.path.exists(path):
        pytest.skip("device assembly not there (build here first)")
    assert isa_check.check_no_parked_registers(open(path).read(), "tile_kernel") == []
