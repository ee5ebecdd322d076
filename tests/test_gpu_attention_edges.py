"""GPU tests of attention over the paged cache at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

from tests.serve_util import DTYPES, Cache, gpu, starts

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L


def attend(c, cu, q, most, **kw):
    return L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), most, **kw)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 40, 2 ** 63 - 2, 2 ** 63 - 1])
@pytest.mark.parametrize("rows,lens", [([9, 3], [5, 40]), ([1, 1], [0, 300]), ([50, 20], [11, 200])])
def test_the_widest_windows_hide_nothing(rows, lens, window):
    """Also for sequences of fewer tokens than rows, the first of which stand before token 0."""
    c, cu = Cache(3, lens, 1, 64, 16), starts(rows)
    q = torch.from_numpy(np.random.default_rng(4).standard_normal((sum(rows), 4, 64))).bfloat16()
    want = attend(c, cu, q, max(rows), softmax_scale=0.2)
    got = attend(c, cu, q, max(rows), softmax_scale=0.2, window=window)
    assert torch.isfinite(want[1]).any() and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
