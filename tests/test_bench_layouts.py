"""Kernel names of the grouped product whose weight layout is a number, as the benchmark
reads them."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


@pytest.mark.parametrize("name,flags", [
    ("_ZN3moe13k_expert_gemmIDF16_Lb1ELb1ELi1ELb0EEEvNS_8GemmArgsE", (True, True, True)),
    ("_ZN3moe13k_expert_gemmIDF16bLb0ELb0ELi0ELb0EEEvNS_8GemmArgsE", (False, False, False)),
    ("void moe::k_expert_gemm<_Float16, true, true, 1, true>(moe::GemmArgs)", (True, True, True)),
    ("void moe::k_expert_gemm<float, true, false, 0, false>(moe::GemmArgs)", (True, False, False)),
])
def test_layouts_in_names(name, flags):
    assert bench.gemm_flags(name) == flags
    short = "k_expert_gemm/" + ("gateup" if flags[0] else "down")
    assert bench.kernel_short_name(name) == short + ("" if flags[2] else "_rowmajor")


def test_the_cells_sources_are_in_the_record_s_hash():
    assert "mixture_experts_routed_amd/csrc/ffn_cells.hpp" in bench.GEMM_SOURCES
