"""CPU checks of the token-serving C ABI at the ends of its ranges, before any HIP call (pointers are fake)."""
import numpy as np
import pytest
import torch

from tests.test_serve_abi_cpu import ARG, DEV, SHAPE, attend, int4

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="valid arguments are passed with fake pointers")


@no_gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_softmax_scales_whose_log2_leaves_fp32(sign):
    """Scores are kept times log2(e): a scale that is finite only without it would make every score infinite or NaN."""
    last = float(np.float32(np.finfo(np.float32).max / 1.4426950408889634))
    assert attend(scale=sign * 0.999 * last) == DEV
    assert attend(scale=sign * 1.001 * last) == ARG and attend(scale=sign * 3.4e38) == ARG
