"""The gradient of the router logits adds the picks' term through LDS that the
lanes of one wavefront share: one lane zeroes a word, another adds to it, the
first reads it back. The hardware keeps a wavefront's LDS operations in order;
the compiler keeps it only where the code says so (a lane that adds nothing
could have its own zero forwarded to its read). Read from the compiler's
intermediate form of this repository's kernel, no GPU."""
import os
import re
import subprocess

import pytest

from mixture_experts_routed_amd import build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """kernel symbol -> its LDS operations in order: Z stores of zero, A atomic adds,
    L loads, F fences of the wavefront"""
    out = str(tmp_path_factory.mktemp("ir") / "balance.ll")
    cmd = [build.hipcc(), *[f for f in build.FLAGS if f not in ("-fPIC", "-Wall")], "-S",
           "-emit-llvm", "--cuda-device-only", os.path.join(build.CSRC, "balance.hip"), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    found, name = {}, None
    for line in open(out):
        m = re.match(r"define .*@(\w+)\(", line)
        if m:
            name = m.group(1)
            found[name] = ""
        elif line.startswith("}"):
            name = None
        elif name:
            lds = "addrspace(3)" in line
            if re.match(r'\s*fence syncscope\("wavefront', line):
                found[name] += "F"
            elif lds and re.match(r"\s*store float 0\.0", line) or lds and "zeroinitializer" in line:
                found[name] += "Z"
            elif lds and "atomicrmw" in line:
                found[name] += "A"
            elif lds and re.search(r"= load ", line):
                found[name] += "L"
    return {k: v for k, v in found.items() if "k_route_backward" in k}


def test_zero_add_and_read_back_are_ordered(kernels):
    assert len(kernels) == 3 * 14  # types; widths
    for name, ops in kernels.items():
        # before a row's zeroing (the reads of the row before), before the adds, before the reads
        assert re.fullmatch(r"F+Z+F+A+F+L+", ops), (name, ops)
