"""Kernel names of the grouped product over 4-bit weights, as the benchmark reads them:
apart from each other and from the kernels of the other layouts."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


@pytest.mark.parametrize("name,flags,short", [
    ("_ZN3moe13k_expert_gemmIDF16_Lb1ELb1ELi2ELb0EEEvNS_8GemmArgsE", (True, True, 2),
     "k_expert_gemm/gateup_mx4"),
    ("_ZN3moe13k_expert_gemmIDF16bLb0ELb0ELi2ELb0EEEvNS_8GemmArgsE", (False, False, 2),
     "k_expert_gemm/down_mx4"),
    ("void moe::k_expert_gemm<_Float16, true, false, 2, false>(moe::GemmArgs)", (True, False, 2),
     "k_expert_gemm/gateup_mx4"),
    ("void moe::k_expert_gemm<__bf16, true, true, 2, true>(moe::GemmArgs)", (True, True, 2),
     "k_expert_gemm/gateup_mx4"),
    ("void moe::k_expert_gemm<__bf16, false, false, 2, false>(moe::GemmArgs)", (False, False, 2),
     "k_expert_gemm/down_mx4"),
])
def test_four_bit_layers(name, flags, short):
    assert bench.gemm_flags(name) == flags
    assert bench.gemm_is_gateup(name) == flags[0]
    assert bench.kernel_short_name(name) == short


@pytest.mark.parametrize("name,layout", [
    ("void moe::k_expert_gemm<_Float16, true, true, true>(moe::GemmArgs)", 1),
    ("void moe::k_expert_gemm<_Float16, true, true, false>(moe::GemmArgs)", 0),
    ("_ZN3moe13k_expert_gemmIfLb1ELb0ELb1EEEvNS_8GemmArgsE", 1),
    ("void moe::k_expert_gemm<float, false, false, 0, false>(moe::GemmArgs)", 0)])
def test_the_other_layouts_keep_their_numbers(name, layout):
    flags = bench.gemm_flags(name)
    assert flags[2] == layout and type(flags[2]) is int


def test_a_name_that_cannot_be_read_is_no_other_kernel_s():
    name = "void moe::k_expert_gemm<_Float16, true, true, 7, false>(moe::GemmArgs)"
    assert bench.gemm_flags(name) is None and not bench.gemm_is_gateup(name)
    assert bench.kernel_short_name(name) not in (
        f"k_expert_gemm/{p}{s}" for p in ("gateup", "down") for s in ("", "_rowmajor", "_mx4"))
