"""CPU audit of the loads into LDS of the linears with an epilogue (no GPU): block_dma_audit.hip calls the address functions
of csrc/gemm_tiles.hpp that the kernels call, for the forms that test_dma_audit.py does not know (fp8r's hand-ordered loop
with a partial last stage, nvfp4 with K % 256 != 0 and its block scales through registers); planted mistakes (in a copy of
the header, on the CPU) make it fail."""
import os
import re
import subprocess

import pytest

from tests.test_dma_audit import CSRC, HIPCC, ROOT

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


def build_and_run(tmp_path, include_dir):
    exe = str(tmp_path / "block_dma_audit")
    tests = os.path.join(ROOT, "tests")
    cmd = [HIPCC, "-std=c++17", "-O1", "-x", "hip", "--cuda-host-only", "-I" + include_dir, "-I" + CSRC,
           "-I" + os.path.join(ROOT, "include"), "-I" + tests, os.path.join(tests, "block_dma_audit.hip"), "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=600)


def test_every_load_of_the_linears_with_an_epilogue_is_in_bounds(tmp_path):
    r = build_and_run(tmp_path, CSRC)
    assert r.returncode == 0, r.stdout[-2000:]
    assert "all loads of the linears with an epilogue in bounds" in r.stdout
    for family in ("fp8 any K 128x128", "fp8 any K 256x192", "fp8 any K 256x256", "w4a4 any K 64x64", "w4a4 any K 128x128",
                   "w4a4 any K 256x192", "fp8 64x64 ring 4", "w4a4 64x128"):
        assert re.search(r"^ok %s" % family, r.stdout, re.M), family


@pytest.mark.parametrize("header,old,new,what", [
    ("gemm_tiles.hpp", "const int voff = (kb + c * Rg::VPC < K) ? lrow * stride + (c << 4) : kOutOfRange;",
     "const int voff = lrow * stride + (c << 4);", "past K"),
    ("gemm_tiles.hpp", "at = kt * (C::KSTAGE / 16), left = ks - at;", "at = kt * (C::KSTAGE / 16), left = 16;", "scales past K"),
    ("gemm_tiles.hpp", "left > 0 && r < BM + BN && row < (w ? N : M);", "left > 0 && r < BM + BN;", "rows past the matrix"),
    ("gemm_tiles.hpp", "C::SB_OFF + 16 * (r - BN)) : -1", "C::SB_OFF + 16 * r) : -1", "LDS place"),
    ("gemm_tiles.hpp", "(int64_t)row * ks + at, there", "(int64_t)row * 16 + at, there", "row pitch"),
])
def test_planted_mistakes_are_caught(tmp_path, header, old, new, what):
    mdir = tmp_path / "mutant"
    mdir.mkdir()
    with open(os.path.join(CSRC, header)) as f:
        text = f.read()
    assert old in text
    (mdir / header).write_text(text.replace(old, new))
    r = build_and_run(tmp_path, str(mdir))
    assert r.returncode != 0 and "VIOLATION" in r.stdout, (what, r.stdout[-500:])


def test_the_kernels_take_their_addresses_from_the_audited_functions():
    with open(os.path.join(CSRC, "gemm_w4a4_tile.hpp")) as f:
        text = f.read()
    body = re.search(r"struct ScaleRows \{.*?\n\};", text, re.S).group(0)
    assert body.count("scale_row_load<BM, BN>(tid + j * kThreads") == 2
    assert not re.search(r"a\.(?:ws|xs)\b(?!\) \+ l\.from| : a\.xs\) \+ l\.from)", body)
