"""The sources of a transformer block's operators compile without a warning."""
import os
import subprocess

import pytest

from block_scaled_precision_row_amd import build


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", ["block_norm.hip", "rope.hip", "gemm_fp8_epilogue.hip", "gemm_w4a4_epilogue.hip",
                                    "gemm_w4a4_any_epilogue.hip", "bsq_block.cpp"])
def test_no_warnings(source):
    r = subprocess.run([build.HIPCC] + build.FLAGS + ["--cuda-device-only"] * source.endswith(".hip")
                       + ["-fsyntax-only", os.path.join(build.CSRC, source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    # (-packed-fp32-ops is no feature of the host compiler, which says so, as it does of options that only links take)
    said = [line for line in r.stderr.splitlines() if "warning:" in line and "packed-fp32-ops" not in line
            and "unused during compilation" not in line]
    assert said == []
