"""The nvfp4 linears with an epilogue at K % 256 != 0 mix their inline-assembly LDS DMA with ordinary loads, and their large
tiles spill SGPRs: the check of test_asm_hazards.py, and that a planted hazard in this very assembly is found."""
import os
import re
import subprocess

import pytest

from block_scaled_precision_row_amd import build
from tests.test_asm_hazards import find_hazards


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
def test_no_stale_operands(tmp_path):
    out = str(tmp_path / "k.s")
    src = os.path.join(build.CSRC, "gemm_w4a4_any_epilogue.hip")
    r = subprocess.run([build.HIPCC] + build.FLAGS + ["--cuda-device-only", "-S", src, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    assert text.count("buffer_load_dwordx4") > 16
    assert find_hazards(text) == []
    # an operand of the first DMA restored from a spill right in front of it
    m = re.search(r";;#ASMSTART\n\s*buffer_load_dwordx4 .*?, (s\d+) offen lds", text)
    planted = text[:m.start()] + "v_readlane_b32 %s, v0, 0\n\t" % m.group(1) + text[m.start():]
    assert find_hazards(planted)

