"""CPU checks of the token-serving C ABI at the ends of its ranges, before any HIP call (pointers are fake)."""
import os

import numpy as np
import pytest
import torch

from tests.test_serve_abi_cpu import ARG, DEV, SHAPE, attend, int4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid arguments are passed with fake pointers")


@no_gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_softmax_scales_whose_log2_leaves_fp32(sign):
    """Scores are kept times log2(e): a scale that is finite only without it would make every score infinite or NaN."""
    last = float(np.float32(np.finfo(np.float32).max / 1.4426950408889634))
    assert attend(scale=sign * 0.999 * last) == DEV
    assert attend(scale=sign * 1.001 * last) == ARG and attend(scale=sign * 3.4e38) == ARG


@no_gpu
def test_the_largest_int4_shapes():
    """N <= 2^27 - 16 and M <= 2^20 - 16, as the header says, and nothing above."""
    n, m = (1 << 27) - 16, (1 << 20) - 16
    assert int4(N=n, ldy=n) == DEV and int4(N=n + 1, ldy=n + 8) == SHAPE
    assert int4(M=m) == DEV and int4(M=m + 1) == SHAPE
    with open(os.path.join(ROOT, "include", "bsq_serve.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    assert "M <= 2^20 - 16, N <= 2^27 - 16, K <= 2^20" in text
