"""GPU tests of the paged cache's operators with starts (cu_seqlens) that do not rise: which rows are written is not
defined, but nothing outside the tensors is, and the call returns as ever."""
import numpy as np
import pytest
import torch

from tests.serve_util import Cache, gpu

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L

STARTS = [[0, 1000, 1200, 100, 150], [0, 40, 3, 900, 1200], [5, 2, 1, 0, 0], [1200, 900, 300, 100, 0],
          [0, 1200, 0, 1200, 0], [-7, 2 ** 31 - 1, -2 ** 31, 64, 2 ** 30]]


def framed(shape, dtype):
    """A tensor with room before and behind it, and the whole of it; every element holds a pattern."""
    n = int(np.prod(shape))
    base = torch.full((n + 8192,), 7, dtype=dtype, device="cuda")
    return base[4096:4096 + n].view(shape), base


def frame_is_whole(base):
    return bool(torch.all(base[:4096] == 7)) and bool(torch.all(base[-4096:] == 7))


@pytest.mark.parametrize("cu", STARTS)
@pytest.mark.parametrize("H,Hq,D", [(2, 8, 64), (1, 20, 128), (2, 2, 64)])
@pytest.mark.parametrize("most", [1, 3, 1200])
def test_starts_that_fall(cu, H, Hq, D, most):
    T, page = 1200, 16
    c = Cache(3, [1300, 700, 1210, 400], H, D, page)
    start = gpu(np.array(cu, np.int64).astype(np.int32))
    lens, table = gpu(c.lens), gpu(c.table)
    pools = [framed(a.shape, gpu(a).dtype) for a in (c.kc, c.vc, c.ks, c.vs)]
    for (t, _), a in zip(pools, (c.kc, c.vc, c.ks, c.vs)):
        t.copy_(gpu(a))
    pools[2][0][::3] = float("nan")                       # scales that a page has before its first token
    pools[3][0][::3] = float("nan")
    kc, vc, ks, vs = (t for t, _ in pools)
    rng = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(T, H, D, generator=rng, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, Hq, D, generator=rng, device="cuda").bfloat16()
    (out, whole_out), (y, whole_y), (lse, whole_lse) = (framed(s, d) for s, d in (
        ((T, Hq, D), torch.bfloat16), ((Hq, T, D), torch.bfloat16), ((T, Hq), torch.float32)))
    n = L.bsq_attention_kv8_workspace_bytes(4, T, most, Hq, H, D)
    ws, whole_ws = framed((max(n, 256),), torch.uint8)
    w = L.bsq_rope_inv_freq(D, 10000.0)[0].cuda()
    for narrow in (False, True):
        L.bsq_kv_append(k, v, start, lens, table, kc, vc, ks, vs, w, q=q, q_out=out)
        ks.nan_to_num_(0.25), vs.nan_to_num_(0.25)
        tab = table if narrow else torch.cat([table, torch.full((4, 1 << 14), -1, dtype=torch.int32, device="cuda")], 1)
        L.bsq_attention_kv8(q, start, lens, tab, kc, vc, ks, vs, most, softmax_scale=0.1, y=y.transpose(0, 1), lse=lse,
                            workspace=ws)
    torch.cuda.synchronize()
    for base in [b for _, b in pools] + [whole_out, whole_y, whole_lse, whole_ws]:
        assert frame_is_whole(base)
