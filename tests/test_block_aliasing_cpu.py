"""A linear's residual may be its output (include/bsq_block.h), so no code that a linear with an epilogue runs through may
promise the compiler that the output is reached by one pointer alone. The plain linears' tiles keep that promise."""
import os
import re
import subprocess

import pytest

from block_scaled_precision_row_amd import build

CHECK = """
#include "epilogue.hpp"
#include "gemm_fp8_tile.hpp"
using namespace bsq;
static_assert(std::is_same<fp8::OutputOf<gemm::TileEpilogue<0>>, uint16_t*>::value, "with an epilogue");
static_assert(std::is_same<fp8::OutputOf<gemm::NoFinish>, uint16_t* __restrict__>::value, "without one");
"""


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="hipcc not available")
def test_only_plain_tiles_promise_an_output_of_their_own(tmp_path):
    src = tmp_path / "check.hip"
    src.write_text(CHECK)
    r = subprocess.run([build.HIPCC] + build.FLAGS + ["--cuda-host-only", "-fsyntax-only", str(src)], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("source,functions", [
    ("gemm_fp8_tile.hpp", ["fp8_tile"]), ("gemm_fp8_epilogue.hip", ["gemm_fp8_epilogue_kernel"]),
    ("gemm_w4a4_tile.hpp", ["w4a4_tile"]), ("gemm_w4a4_epilogue.hpp", ["gemm_w4a4_epilogue_kernel"]),
    ("gemm_skinny.hip", ["gemm_skinny_epilogue_kernel", "gemm_skinny_staged_epilogue_kernel", "skinny_epilogue"]),
    ("epilogue.hpp", ["epilogue_tile", "load_tile_rows"])])
def test_no_restricted_output_or_residual(source, functions):
    with open(os.path.join(build.CSRC, source)) as f:
        text = f.read()
    for name in functions:
        head = re.search(r"void\s+%s\((.*?)\)\s*(?:const\s*)?\{" % name, text, re.S).group(1)
        assert not re.search(r"__restrict__\s+(?:y|r|residual|e|a)\b", head), (source, name)
