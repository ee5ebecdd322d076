"""GPU parity tests of rotary positions with several axes against the fp64 oracle (oracle/block.py). The tolerance is
that of one axis: the angle's rest is rounded to fp32 (2^-25 pi absolute) and sine and cosine carry 2 ulp (2^-22); each
output is two products and a sum in fp32: |err| <= f (|a| + |b|) 2^-21, then one rounding u(t)."""
import numpy as np
import pytest
import torch

from oracle import block
from tests.block_util import DTYPES, f64, u

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L


def bound(x, ref, pairs, factor, kind, interleaved):
    m = np.zeros(ref.shape)
    a = np.abs(f64(x))
    first = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    second = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    m[..., first] = m[..., second] = factor * (a[..., first] + a[..., second])
    tiny = 2.0 ** -25 if kind == "fp16" else 0.0
    return np.where(m > 0, u(DTYPES[kind]) * np.abs(ref) + m * 2.0 ** -21 + tiny, 0.0)


def frequencies(pairs):
    return torch.from_numpy(10000.0 ** (-np.arange(pairs) / pairs)).float()


CASES = [
    # tokens, heads, dim, sections, cycled, backward
    (1, 1, 16, [8], False, False),
    (3, 5, 128, [8, 28, 28], False, True),
    (70, 8, 128, [12, 10, 10], True, False),
    (1030, 24, 64, [16, 16], False, False),
    (17, 3, 256, [0, 64, 0, 64], False, True),
    (5, 2, 7, [1, 2], False, False),
    (6, 3, 66, [9, 8], True, True),
    (2, 1, 2, [1], True, False),
    (9, 40, 1024, [128, 128, 128, 128], True, False),
    (2100, 40, 64, [3, 3, 2], True, True),
    (40, 2, 128, [64, 0, 0], True, False),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,sections,cycled,backward", CASES)
def test_rope_axes(T, H, D, sections, cycled, backward, interleaved, kind):
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, H, D))).to(DTYPES[kind])
    pos, w, factor = rng.integers(-50, 5000, (T, len(sections))), frequencies(sum(sections)), 1.25
    ref = block.rope_axes(f64(x), pos, f64(w), sections, cycled, interleaved, factor, backward)
    y = L.bsq_rope_axes(x.cuda(), torch.from_numpy(pos).cuda(), w.cuda(), sections,
                        L.BSQ_AXES_CYCLED if cycled else L.BSQ_AXES_BLOCKS,
                        L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF, factor, backward=backward)
    assert np.all(np.abs(f64(y) - ref) <= bound(x, ref, sum(sections), factor, kind, interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(37, 6, 128, 128), (5, 2, 66, 34), (1100, 24, 64, 32)])
def test_equal_axes_are_bsq_rope(T, H, D, rot, interleaved):
    layout = L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF
    x, pos = torch.randn(T, H, D, device="cuda").bfloat16(), torch.randint(0, 1 << 40, (T,), device="cuda")
    w = frequencies(rot // 2).cuda()
    want = L.bsq_rope(x, pos, w, layout, 0.5)
    n = rot // 2
    for sections, order in (([n], 1), ([n], 2), ([n - n // 3, n // 3], 1), ([n - 2 * (n // 3), n // 3, n // 3], 2)):
        got = L.bsq_rope_axes(x, pos[:, None].expand(T, len(sections)), w, sections, order, layout, 0.5)
        assert torch.equal(got, want)


def test_strides_and_in_place():
    T, H, D, sections = 45, 6, 128, [16, 24, 24]
    x, w = torch.randn(T, H, D, device="cuda").bfloat16(), frequencies(64).cuda()
    pos = torch.randint(0, 999, (T, 3), device="cuda")
    want = L.bsq_rope_axes(x, pos, w, sections)
    planes = pos.t().contiguous().t()                           # a row of positions for each axis
    assert planes.stride() == (1, T) and torch.equal(L.bsq_rope_axes(x, planes, w, sections), want)
    dense = x.clone()
    assert L.bsq_rope_axes(dense, pos, w, sections, y=dense) is dense and torch.equal(dense, want)
    fused = torch.zeros(T, H + 4, D, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:2 + H] = x
    out = torch.full((H, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    L.bsq_rope_axes(fused[:, 2:2 + H], pos, w, sections, y=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want)
    odd = torch.full((T * (H * D + 3) + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(odd, (T, H, D), (H * D + 3, D, 1), 1)
    view.copy_(x)
    L.bsq_rope_axes(view, pos, w, sections, y=view)
    assert torch.equal(view, want) and odd[0] == 7.0
    y = L.bsq_rope_axes(x[:1].expand(T, H, D), pos[:1].expand(T, 3), w, sections)   # one token for all
    assert torch.equal(y, want[:1].expand(T, H, D))


def test_gradient_is_the_transpose():
    """<R x, dy> = <x, R^T dy>: the map is linear, so this is its gradient; fp32, each product off by 2^-20."""
    T, H, D, sections = 9, 3, 64, [12, 10, 10]
    for order, layout in ((1, 1), (2, 2)):
        x, dy = torch.randn(2, T, H, D, device="cuda")
        pos, w = torch.randint(0, 9999, (T, 3), device="cuda"), frequencies(32).cuda()
        y = L.bsq_rope_axes(x, pos, w, sections, order, layout, 1.5)
        dx = L.bsq_rope_axes(dy, pos, w, sections, order, layout, 1.5, backward=True)
        a, b = (f64(y) * f64(dy)).sum(), (f64(x) * f64(dx)).sum()
        assert abs(a - b) <= 2.0 ** -19 * 1.5 * (np.abs(f64(x)).sum() * np.abs(f64(dy)).max())


def test_captured_and_replayed():
    T, H, D, sections = 64, 8, 128, [32, 32]
    x, w = torch.randn(T, H, D, device="cuda").half(), frequencies(64).cuda()
    pos = torch.randint(0, 999, (T, 2), device="cuda")
    L.bsq_rope_axes(x, pos, w, sections)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = L.bsq_rope_axes(x, pos, w, sections)
    for i in range(4):
        x.normal_()
        pos.random_(0, 5000)
        g.replay()
        want = L.bsq_rope_axes(x, pos, w, sections)
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
