"""What the dense product's assembly statements rely on, read from the compiler's
assembly of this repository's kernel (no GPU): where matrix instructions are
written in assembly, the compiler keeps no wait states around them, so no
accumulator may be moved and nothing spilled between them; m0 and the scalar
registers that the loads into LDS pass their resource through belong to them."""
import os
import re
import subprocess

import pytest

from mixture_experts_routed_amd import build


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """kernel symbol -> its instructions, in order"""
    out = str(tmp_path_factory.mktemp("isa") / "linear.s")
    cmd = [build.hipcc(), *[f for f in build.FLAGS if f not in ("-fPIC", "-Wall")], "-S",
           "--cuda-device-only", os.path.join(build.CSRC, "linear.hip"), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    found, name = {}, None
    for line in open(out):
        m = re.match(r"^(_Z\w+):", line)
        if m:
            name = m.group(1)
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name and (line.startswith("\t") and not line.startswith("\t.") or line[0] == "."):
            text = line.split(";")[0].strip()
            if text and not text.endswith(":"):
                found[name].append(text)
    return {k: v for k, v in found.items() if "k_gemm" in k}


def test_large_tile_kernels(kernels):
    large = {k: v for k, v in kernels.items() if "Li256ELi256E" in k}
    assert len(large) == 6  # two types, three operand forms
    for name, code in large.items():
        at = [i for i, t in enumerate(code) if t.startswith("v_mfma")]
        assert len(at) == 64, name  # four k-groups of 16, once
        loop = code[at[0]:at[-1] + 1]
        for t in loop:
            assert not t.startswith(("v_accvgpr", "scratch_")), (name, t)
        # operands come from LDS reads: whatever last wrote one before its matrix
        # instruction (around the loop's end too) is no vector arithmetic
        writer = {}
        for t in loop + loop:
            if t.startswith("v_mfma"):
                a = re.findall(r"v\[(\d+):(\d+)\]", t)
                assert len(a) == 2 and t.count("a[") == 2, t  # accumulators: accumulation registers
                for lo, hi in a:
                    for r in range(int(lo), int(hi) + 1):
                        assert writer.get(r, "ds_read").startswith("ds_read"), (name, t, writer[r])
                continue
            m = re.match(r"((?:v|ds_read)\w+) v\[?(\d+)(?::(\d+))?", t)
            if m:
                for r in range(int(m.group(2)), int(m.group(3) or m.group(2)) + 1):
                    writer[r] = t


def test_loads_into_lds_own_their_scalar_registers(kernels):
    assert len(kernels) >= 6 + 9
    for name, code in kernels.items():
        for t in code:
            if re.search(r"\bm0\b", t):
                assert t.startswith("s_mov_b32 m0, "), (name, t)
        loads = [i for i, t in enumerate(code) if t.startswith("buffer_load") and t.endswith("lds")]
        for i in loads:
            assert code[i].split(", ")[1] == "s[96:99]", (name, code[i])
            assert code[i - 3].startswith("s_mov_b32 m0") and all(
                code[i - k].startswith("s_mov_b64 s[9") for k in (1, 2)), (name, code[i - 3:i + 1])
