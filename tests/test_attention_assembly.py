"""The attention kernels multiply their accumulators in place in a line of assembly, before which the
compiler keeps no distance from the matrix products that write them.  In the assembly of this
library's own source, every such line comes behind enough wait states, with no product in between."""

import os
import re
import subprocess

import pytest

from precision_gemm_amd import build as B

# between a product of 16 passes and an instruction that reads or writes its result
WAITS = 20


def test_accumulators_are_settled(tmp_path):
    try:
        hipcc = B.hipcc()
    except Exception as e:  # pragma: no cover
        pytest.skip(str(e))
    out = str(tmp_path / "tree.s")
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC") and not f.startswith("-Rpass")]
    subprocess.run([hipcc, *flags, "--cuda-device-only", "-S", os.path.join(B.CSRC_ATTN, "tree_attention.hip"), "-o", out],
                   check=True, capture_output=True)
    in_asm = False
    waits, kernels, found = 0, set(), 0
    kernel = ""
    for line in open(out):
        line = line.strip()
        m = re.match(r"(_Z\w+):", line)
        if m:
            kernel = m.group(1)
        if line.endswith(":") or re.match(r"[.\w$]+:", line):  # a label: other ways lead here
            waits = 0
        elif line.startswith(";;#ASMSTART"):
            in_asm = True
        elif line.startswith(";;#ASMEND"):
            in_asm = False
        elif line.startswith("v_mfma"):
            waits = 0
        elif line.startswith("s_nop") and in_asm:
            waits += int(line.split()[1]) + 1
        elif line.startswith("v_mul_f32 ") and in_asm:
            assert waits >= WAITS, f"{kernel}: {line}"
            found += 1
            kernels.add(kernel)
    # eighteen forms of the two attention kernels, each with four tiles of four values at least
    assert len(kernels) == 18 and found >= 16 * len(kernels), (len(kernels), found)
