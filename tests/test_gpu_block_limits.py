"""GPU tests of the block norms at the row counts where a launch of a workgroup a row would end.

Rows of +-1 with eps 0 have N(v) = v in both their sums (16 squares of 1, 1 / sqrt(1)), and dy of -1, 0 and 1 makes every
partial sum of the vectors' gradients a whole number below 2^24: they are exact in fp32, in any order."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L

D = 16


def rows_of_signs(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(0, 2, (T, D), dtype=torch.int8, device="cuda", generator=g).mul_(2).sub_(1).bfloat16()
    dy = torch.randint(-1, 2, (T, D), dtype=torch.int8, device="cuda", generator=g).bfloat16()
    return x, dy


def sums(t):
    """Whole-number sums of the columns, by pieces."""
    return sum(p.sum(0, dtype=torch.float64) for p in t.split(1 << 22))


def test_gradient_of_more_rows_than_a_launch_has_workgroups():
    T = (1 << 26) + 77                                            # a forward launch ends at 2^25 rows
    x, dy = rows_of_signs(T, 1)
    w, b = torch.ones(2, D, dtype=torch.bfloat16, device="cuda")
    st = torch.tensor([0, 5, 1 << 25, T - 9], dtype=torch.int32, device="cuda")
    scale = torch.zeros(3, D, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    out = L.bsq_block_norm_backward(dy, None, x, norm=L.BSQ_NORM_RMS, eps=0.0, weight=w, bias=b, scale=scale, starts=st, dx=dx)
    live = slice(0, T - 9)
    n = sum((p.double() * q.double()).sum(0) for p, q in zip(x[live].split(1 << 22), dy[live].split(1 << 22)))
    assert torch.equal(out["weight"].double(), n)
    assert torch.equal(out["bias"].double(), sums(dy[live]))
    for g, (a, e) in enumerate(((0, 5), (5, 1 << 25), (1 << 25, T - 9))):
        want = sum((p.double() * q.double()).sum(0) + q.double().sum(0)          # dy (n weight + bias)
                   for p, q in zip(x[a:e].split(1 << 22), dy[a:e].split(1 << 22)))
        assert torch.equal(out["scale"][g].double(), want), g
    assert torch.all(dx[T - 9:] == 7.0)
    for a in range(0, T - 9, 1 << 22):                            # rows are independent: those of small calls
        e = min(a + (1 << 22), T - 9)
        part = L.bsq_block_norm_backward(dy[a:e], None, x[a:e], norm=L.BSQ_NORM_RMS, eps=0.0, weight=w, bias=b, need=("x",))
        assert torch.equal(dx[a:e], part["x"]), a


def test_most_rows_of_a_forward_launch():
    T = (1 << 25) - 5
    x = rows_of_signs(T, 2)[0]
    w = torch.linspace(-2, 2, D, device="cuda").bfloat16()
    y = L.bsq_block_norm(x, norm=L.BSQ_NORM_RMS, eps=0.0, weight=w)[0]
    assert torch.equal(y, x * w)
    with pytest.raises(L.BsqError):
        L.bsq_block_norm(x[:1].expand(T + 1, D), norm=L.BSQ_NORM_RMS, weight=w)
