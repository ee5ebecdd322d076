"""The attention kernels load tiles into LDS by inline assembly: no SGPR operand of it (M0 included) may have been
written by a VALU instruction within five wait states, as test_asm_hazards.py explains and checks for the GEMMs."""
import os

import pytest

from tests.test_asm_hazards import find_hazards
from block_scaled_precision_row_amd import build
import subprocess


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("source", ["kv_attn.hip", "kv_prompt.hip"])
def test_no_stale_operands(source, tmp_path):
    out = str(tmp_path / "k.s")
    r = subprocess.run([build.HIPCC] + build.FLAGS + ["--cuda-device-only", "-S", os.path.join(build.CSRC, source), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    assert text.count("global_load_lds_dwordx4") > 16
    assert find_hazards(text) == []
