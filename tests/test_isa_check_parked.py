"""What the build's check of the 8-bit head's tile kernels takes for a register parked in
an accumulator, form by form (CPU only)."""

import os

import pytest

from rollout_logprob_consistency_amd import isa_check

KERNEL = """
_ZN2lp11tile_kernelE:
	v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], 0
	v_mfma_i32_16x16x64_i8 a[0:3], v[0:3], v[4:7], a[0:3]
%s
	v_accvgpr_read_b32 v8, a0
	v_add_u32_e32 v9, v8, v7
.Lfunc_end0:
_ZN2lp13stream_kernelE:
	v_accvgpr_mov_b32 a0, a1
.Lfunc_end1:
"""


def problems(line):
    return isa_check.check_no_parked_registers(KERNEL % ("\t" + line), "tile_kernel")


@pytest.mark.parametrize("line", [
    "v_accvgpr_write_b32 a5, v218", "v_accvgpr_write_b32 a5, 0", "v_accvgpr_mov_b32 a7, a200",
    "ds_read_b32 a3, v12", "ds_read_b128 a[4:7], v9 offset:64",
    "ds_read2st64_b64 a[0:3], v9 offset0:1", "buffer_load_dword a9, v1, s[0:3], 0 offen",
    "buffer_load_dwordx4 a[8:11], v1, s[0:3], 0 offen", "global_load_dwordx2 a[2:3], v[0:1], off",
    "flat_load_dword a1, v[0:1]", "global_atomic_add a2, v[0:1], v3, off sc0",
    "scratch_store_dword off, v0, off", "scratch_load_dword v0, off, off",
    "scratch_store_dwordx2 off, a[0:1], s33", "v_mov_b32_e32 a4, v1 ; a comment"])
def test_planted_ones_are_found(line):
    found = problems(line)
    assert len(found) == 1 and "tile_kernel" in found[0] and ": 1 " in found[0]


@pytest.mark.parametrize("line", [
    "v_mfma_i32_16x16x64_i8 a[4:7], v[0:3], v[4:7], a[0:3]", "v_accvgpr_read_b32 v1, a7",
    "buffer_store_dword a0, v1, s[0:3], 0 offen", "ds_write_b32 v0, a3",
    "ds_read_b128 v[4:7], v9", "buffer_load_dwordx4 v1, s[0:3], 0 offen lds", "s_add_u32 s0, s1, s2",
    "s_barrier", "; v_accvgpr_write_b32 a0, v1", ".LBB0_1:", "v_add_u32_e32 v1, v2, v3"])
def test_others_are_not(line):
    assert problems(line) == []


def test_the_built_kernels():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "_build",
                        "int8.device.s")
    if not os.path.exists(path):
        pytest.skip("device assembly not there (build here first)")
    text = open(path).read()
    assert isa_check.check_no_parked_registers(text, "tile_kernel") == []
    # (The check sees the forms that this compiler uses where they are.)
    assert "v_accvgpr_mov_b32" not in text or \
        isa_check.check_no_parked_registers(text, "stream_kernel")
