"""What the linear cross entropy kernel asks of the compiler, on the CPU."""

import os
import re
import subprocess

import pytest

from learned_optimizer_step_gb300 import build as B

SOURCE = os.path.join(B.CSRC, "k_linear_ce.cu")


def test_the_kernel_has_the_registers_that_its_warps_share_out(tmp_path):
    """Its first warpgroup gives registers to the two of the epilogue, which would wait for
    them for ever if the launch had fewer than the source counts on: the library refuses the
    call then, so that a build with another count has to be noticed before."""
    try:
        nvcc = B._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    want = int(re.search(r"kRegs = (\d+)", open(SOURCE).read()).group(1))
    r = subprocess.run([nvcc] + B.NVCC_FLAGS + ["-Xptxas", "-v", "-c", SOURCE, "-o", str(tmp_path / "k.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    said = re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", r.stderr, re.S)
    got = [int(n) for name, n in said if "11k_linear_ceE" in name]
    assert got == [want], said
