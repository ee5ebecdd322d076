"""Pins of oracle/block.py: closed values, invariants and differences."""
import math

import numpy as np
import pytest

from oracle import block, serve


def test_axes_by_hand():
    assert block.axis_of_pairs([2, 0, 3], False) == [0, 0, 2, 2, 2]
    assert block.axis_of_pairs([4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    assert block.axis_of_pairs([3, 1], True) == [0, 1, 0, 0]
    assert block.axis_of_pairs([5], True) == [0] * 5


@pytest.mark.parametrize("interleaved", [False, True])
def test_equal_positions_are_one_axis(interleaved):
    rng = np.random.default_rng(0)
    x, p, w = rng.standard_normal((5, 2, 20)), rng.integers(0, 100, 5), rng.random(8)
    for sections, cycled in (([3, 5], False), ([4, 2, 2], True)):
        y = block.rope_axes(x, np.stack([p] * len(sections), 1), w, sections, cycled, interleaved, 1.5)
        assert np.allclose(y, serve.rope(x, p, w, interleaved, 1.5), rtol=0, atol=1e-14)


def test_each_axis_turns_its_own_pairs():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((1, 1, 12)), np.array([0.5, 0.25, 0.125, 1.0, 2.0, 3.0])
    p = np.array([[3, 7, 11]])
    y = block.rope_axes(x, p, w, [1, 2, 3])
    for i, c in enumerate([0, 1, 1, 2, 2, 2]):
        z = complex(x[0, 0, i], x[0, 0, i + 6]) * np.exp(1j * p[0, c] * w[i])
        assert abs(complex(y[0, 0, i], y[0, 0, i + 6]) - z) < 1e-13


def test_norms_of_known_rows():
    n, r = block.normed(np.array([[3.0, -3.0, 3.0, -3.0]]), "rms", 0.0)
    assert np.allclose(n, [[1, -1, 1, -1]]) and np.allclose(r, 1 / 3)
    n, _ = block.normed(np.array([[5.0, 7.0]]), "layer", 0.0)
    assert np.allclose(n, [[-1, 1]])
    rng = np.random.default_rng(2)
    v = rng.standard_normal((3, 40))
    assert np.allclose(block.normed(4 * v + 9, "layer", 0.0)[0], block.normed(v, "layer", 0.0)[0])
    assert np.allclose(block.normed(4 * v, "rms", 0.0)[0], block.normed(v, "rms", 0.0)[0])
    assert np.allclose((block.normed(v, "layer", 0.0)[0] ** 2).mean(-1), 1)
    assert np.all(block.normed(np.zeros((1, 4)), "layer", 1e-6)[0] == 0)


CASES = [
    dict(norm="layer"), dict(norm="rms", weight=1), dict(norm="layer", weight=1, bias=1, scale=1, shift=1),
    dict(norm="rms", scale=1, branch=1, gate=1), dict(norm="layer", shift=1, branch=1, gate=1, post="rms", post_weight=1),
    dict(norm=None, branch=1, gate=1, post="layer"), dict(norm="rms", weight=1, branch=1, post="rms", post_weight=1),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_gradient_against_differences(case):
    rng = np.random.default_rng(3)
    T, D, groups, starts = 7, 12, 3, [0, 2, 2, 6]
    group = block.group_of_rows(T, groups, starts)
    assert group.tolist() == [0, 0, 2, 2, 2, 2, -1]
    shapes = {"x": (T, D), "branch": (T, D), "weight": (D,), "bias": (D,), "post_weight": (D,), "scale": (groups, D),
              "shift": (groups, D), "gate": (groups, D)}
    v = {k: rng.standard_normal(s) if k == "x" or case.get(k) else None for k, s in shapes.items()}
    fixed = dict(norm=case["norm"], eps=1e-3, post=case.get("post"), post_eps=1e-2, group=group)
    live = (group >= 0)[:, None]
    dy, do = rng.standard_normal((T, D)) * live, rng.standard_normal((T, D)) * live

    def total(v):
        o, y = block.block_norm(**v, **fixed)
        return (o * do).sum() + (0.0 if y is None else (y * dy).sum())

    x_out = block.block_norm(**v, **fixed)[0]
    back = {k: v[k] for k in v if k != "x"}
    grads = block.block_norm_backward(dy if case["norm"] else None, do, x_out, **back, **fixed, groups=groups)
    for k in v:
        if v[k] is None:
            continue
        d = rng.standard_normal(v[k].shape)
        if k in ("x", "branch"):
            d = d * live
        h = 1e-5
        up, down = dict(v), dict(v)
        up[k], down[k] = v[k] + h * d, v[k] - h * d
        diff = (total(up) - total(down)) / (2 * h)
        assert abs(diff - (grads[k] * d).sum()) <= 1e-7 * (1 + abs(diff)), k


def test_activations():
    v = np.linspace(-9, 9, 1001)
    assert block.activation(0.0, "silu") == 0 and block.activation(0.0, "gelu") == 0
    assert np.allclose(block.activation(v, "silu") - block.activation(-v, "silu"), v)
    for act in ("gelu", "gelu_tanh"):
        assert np.allclose(block.activation(v, act) - block.activation(-v, act), v)
    tanh = 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    assert np.allclose(block.activation(v, "gelu_tanh"), tanh, rtol=0, atol=1e-15 * 9)
    assert abs(block.activation(1.0, "silu") - 1 / (1 + math.exp(-1))) < 1e-15
    # v Phi(v), Phi by the trapezoid sum of its density
    t = np.linspace(-12, 1.3, 400001)
    phi = np.trapezoid(np.exp(-t * t / 2), t) / math.sqrt(2 * math.pi)
    assert abs(block.activation(1.3, "gelu") - 1.3 * phi) < 1e-9
    assert np.max(np.abs(block.activation(v, "gelu") - block.activation(v, "gelu_tanh"))) < 1e-3


def test_epilogue_by_hand():
    v = np.array([[1.0, 2.0], [3.0, 4.0]])
    y = block.epilogue(v, bias=np.array([1.0, -2.0]), gate=np.array([[2.0, 3.0], [5.0, 7.0]]),
                       residual=np.array([[10.0, 20.0], [30.0, 40.0]]), group=np.array([1, 0]))
    assert y.tolist() == [[10 + 5 * 2, 20 + 7 * 0], [30 + 2 * 4, 40 + 3 * 2]]
