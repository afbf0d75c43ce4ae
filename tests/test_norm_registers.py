"""CPU test that what the norm's kernels keep in registers stays there: the compiler's report of every one has no scratch memory."""
import os
import re
import subprocess

import pytest

from gated_mlp_gemms_amd import build as B


def test_no_kernel_spills(tmp_path):
    if not os.path.exists(B.HIPCC):
        pytest.skip("the ROCm compilers are not installed")
    r = subprocess.run([B.HIPCC, *B.CFLAGS, "--cuda-device-only", "-Rpass-analysis=kernel-resource-usage", "-c",
                        os.path.join(B.CSRC, "norm.hip"), "-o", str(tmp_path / "norm.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    use = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", r.stderr, re.S)
    assert len(use) > 50 and all("norm_" in name for name, _ in use)
    assert [(name, int(n)) for name, n in use if int(n)] == []
