"""CPU checks of the row limits that include/bsq_block.h states for the block norms, by the argument checks alone: pointers
are fake and never dereferenced; calls with valid arguments are made only where there is no GPU, where they report
BSQ_ERR_DEVICE."""
import pytest

from tests.test_block_abi_cpu import DEV, NO_GPU, SHAPE, A, back
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
