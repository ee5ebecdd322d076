"""GPU tests of attention over the paged cache at the ends of its arguments' ranges."""
import numpy as np
import pytest
import torch

from oracle import serve
from tests.serve_util import DTYPES, Cache, attention_bounds, f64, gpu, starts

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


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens", [([1, 1], [70, 300]), ([3], [90]), ([40], [200])])
def test_a_scale_of_zero_is_a_product_like_any_other(rows, lens, kind):
    """Rows of finite queries take the mean, a row with a NaN or an infinity in its query is NaN (0 times it is)."""
    c, cu = Cache(5, lens, 1, 64, 16), starts(rows)
    q = torch.from_numpy(np.random.default_rng(6).standard_normal((sum(rows), 4, 64))).to(DTYPES[kind])
    want, want_l = attend(c, cu, q, max(rows), softmax_scale=0.0)
    assert torch.isfinite(want).all()
    q[0, 1, 7], q[-1, 2, 40] = float("nan"), float("inf")
    y, lse = attend(c, cu, q, max(rows), softmax_scale=0.0)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    bad[0, 1] = bad[-1, 2] = True
    assert torch.isnan(y.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    assert torch.equal(y.cpu()[~bad], want.cpu()[~bad]) and torch.equal(lse.cpu()[~bad], want_l.cpu()[~bad])


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, 4200), (256, 0)])
def test_long_chunks_of_many_heads(D, window):
    """Blocks for more than half of the compute units, long enough to be cut in two. All heads hold the same: the first
    is checked, the others have to be equal to it."""
    H, rows, lens = 40, [500], [4700]
    c = Cache(D, lens, 1, D, 64)
    q = torch.from_numpy(np.random.default_rng(D + 1).standard_normal((500, 1, D))).bfloat16()
    dev = [gpu(a) for a in (c.lens, c.table)] + [gpu(a).expand(-1, H, *a.shape[2:]).contiguous() for a in (c.kc, c.vc, c.ks, c.vs)]
    y, lse = L.bsq_attention_kv8(q.cuda().repeat(1, H, 1), gpu(starts(rows)), *dev, 500, window=window)
    ref, rl, parts = serve.attention(f64(q), starts(rows), c.lens, *c.host(), D ** -0.5, window)
    ty, tl = attention_bounds(ref, rl, parts, q.dtype, D)
    assert np.all(np.abs(f64(y[:, :1]) - ref) <= ty) and np.all(np.abs(f64(lse[:, :1]) - rl) <= tl)
    assert torch.equal(y, y[:, :1].repeat(1, H, 1)) and torch.equal(lse, lse[:, :1].repeat(1, H))
