"""The linears with an epilogue load their tiles into LDS by inline assembly: no SGPR operand of it (M0 included) may
have been written by a VALU instruction within five wait states, as test_asm_hazards.py explains and checks for the plain
ones."""
import os
import subprocess

import pytest

from block_scaled_precision_row_amd import build
from tests.test_asm_hazards import find_hazards


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", ["gemm_fp8_epilogue.hip", "gemm_w4a4_epilogue.hip"])
def test_no_stale_operands(source, tmp_path):
    out = str(tmp_path / "k.s")
    r = subprocess.run([build.HIPCC] + build.FLAGS + ["--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    assert text.count("buffer_load_dwordx4") > 16
    assert find_hazards(text) == []
