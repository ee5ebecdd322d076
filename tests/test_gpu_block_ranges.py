"""The block norms at both ends of the range that include/bsq_block.h states for their statistics: with eps 0, rows whose
largest element is 2^-56 up to rows of 2^56, in one element or in all. Their tolerances are relative, as elsewhere: a square
of the largest is 2^-112 or more, so what fp32 loses of the others below 2^-149 is at most 16384 x 2^-150 / 2^-112 = 2^-24
of the sum; and a mean of squares of 2^-112 / 16384 is still in fp32's normal range."""
import os
import re

import numpy as np
import pytest
import torch

from oracle import block
from tests.block_util import DTYPES, backward_bounds, f64, forward_bounds, rounded
from tests.test_gpu_block_norm import KINDS

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L


@pytest.mark.parametrize("D", [64, 1032, 16384])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_range_of_the_statistics(kind, norm, D):
    g = torch.Generator().manual_seed(D)
    rows = []
    for e in (-56, -30, 0, 30, 56):
        v = torch.rand(D, generator=g, dtype=torch.float64) * 2 - 1
        v[0], v[1] = 1.0, -1.0                                    # (x - mean reaches the size of x)
        rows.append(v * 2.0 ** e)
        one = torch.zeros(D, dtype=torch.float64)
        one[D // 3] = 2.0 ** e
        rows.append(one)
    x = torch.stack(rows).to(DTYPES[kind])
    T, group = len(x), np.zeros(len(x), dtype=np.int64)
    _, _, y, ey = forward_bounds(f64(x), norm, 0.0, group)
    got = L.bsq_block_norm(x.cuda(), norm=KINDS[norm], eps=0.0)[0]
    assert np.all(np.abs(f64(got) - y) <= ey + rounded(y, DTYPES[kind]) + 2.0 ** -23 * np.abs(y))
    dy = torch.randn(T, D, generator=g, dtype=torch.float64).to(DTYPES[kind])
    ref, tol = backward_bounds(f64(dy), None, f64(x), norm, 0.0, group, 1)
    dx = f64(L.bsq_block_norm_backward(dy.cuda(), None, x.cuda(), norm=KINDS[norm], eps=0.0)["x"])
    # (in units of the row's own 1 / size, so that 2^-126 is nothing beside it)
    r = block.normed(f64(x), norm, 0.0)[1]
    assert np.all(np.abs(dx - ref["x"]) <= tol["x"] + rounded(ref["x"], DTYPES[kind]) + 2.0 ** -23 * r + 2.0 ** -126)
    zero = L.bsq_block_norm(torch.zeros(1, D, device="cuda"), norm=KINDS[norm], eps=0.0)[0]
    assert torch.isnan(zero).all()


def test_header_states_it():
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "bsq_block.h")) as f:
        text = re.sub(r"\s*\n \* ", " ", f.read())
    assert "they overflow where |x| reaches 2^57, and with eps 0 they lose what is below 2^-56" in text
