"""CPU checks of the row limits that include/bsq_block.h states for the block norms, by the argument checks alone: pointers
are fake and never dereferenced; calls with valid arguments are made only where there is no GPU, where they report
BSQ_ERR_DEVICE."""
import os
import re

import pytest

from tests.test_block_abi_cpu import DEV, NO_GPU, ROOT, SHAPE, A, back, norm
from block_scaled_precision_row_amd import _lib

MOST = 1 << 30


@pytest.mark.parametrize("dim", [8, 64, 512, 2048, 4096, 16384])
def test_gradient_takes_every_row_count_of_the_header(dim):
    strides = dict(dim=dim, dys=dim, xos=dim, dxs=dim)
    assert back(rows=MOST + 1, **strides) == SHAPE
    need = _lib.bsq_block_norm_workspace_bytes(MOST, dim, 1)
    assert need > 0 and _lib.bsq_block_norm_workspace_bytes(MOST + 1, dim, 1) == 0
    if NO_GPU:
        for rows in (1 << 21, 1 << 23, 1 << 25, MOST):
            assert back(rows=rows, **strides) == DEV, rows
            assert back(rows=rows, weight=A, dw=A, n=need, **strides) == DEV, rows


@pytest.mark.parametrize("dim,waves", [(8, 1), (512, 1), (520, 2), (1024, 2), (2048, 4), (2056, 3), (4096, 4), (4104, 5),
                                       (8192, 8), (16384, 16)])
def test_forward_takes_the_rows_that_the_header_states(dim, waves):
    with open(os.path.join(ROOT, "include", "bsq_block.h")) as f:
        text = re.sub(r"\s*\n \* ", " ", f.read())
    assert ("rows times the waves of a row, ceil(dim / 512) up to dim 2048 and ceil(dim / 1024) above, stay below 2^25 - 4"
            in text)
    assert waves == (-(-dim // 512) if dim <= 2048 else -(-dim // 1024))
    most = -(-((1 << 25) - 4) // waves) - 1                       # the last whose product is below
    strides = dict(dim=dim, xs=dim, ys=dim)
    for rows in (most + 1, MOST):
        assert norm(rows=rows, **strides) == SHAPE, rows
    if NO_GPU:
        assert norm(rows=most, **strides) == DEV
