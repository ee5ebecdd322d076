"""Oracle of the operators around the linears of a transformer block: rotary positions with several axes, the gated
residual with the norms before and after it and its gradient, and the epilogue of a linear.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain fp64 NumPy from the definitions in include/bsq_block.h,
row by row where rows differ; inputs are float64 arrays of exactly representable values.

Pins (``tests/test_oracle_block.py``): axes against rotations by one axis at a time, norms by their invariants (mean,
size, scale and shift of the input), the gradient against differences of the forward, activations by closed values,
symmetries and their definitions' integrals.
"""
import math

import numpy as np

from .serve import rope


def axis_of_pairs(sections, cycled):
    """The axis of each rotated pair."""
    axes, out = len(sections), []
    for i in range(sum(sections)):
        if cycled:
            c = i % axes
            out.append(c if i // axes < sections[c] else 0)
        else:
            c = 0
            while i >= sum(sections[:c + 1]):
                c += 1
            out.append(c)
    return out


def rope_axes(x, positions, inv_freq, sections, cycled=False, interleaved=False, factor=1.0, backward=False):
    """x [T, H, D], positions [T, axes]: each axis' pairs taken from a rotation by that axis alone."""
    y = np.array(x, dtype=np.float64)
    half = sum(sections)
    for c in range(len(sections)):
        by_c = rope(x, np.asarray(positions)[:, c], inv_freq, interleaved, factor, backward)
        for i, a in enumerate(axis_of_pairs(sections, cycled)):
            if a == c:
                for e in ((2 * i, 2 * i + 1) if interleaved else (i, i + half)):
                    y[..., e] = by_c[..., e]
    return y


def group_of_rows(rows, groups, starts=None):
    """The group of each row, -1 for rows behind the last group."""
    out = np.full(rows, -1, dtype=np.int64)
    for g in range(groups):
        if starts is None:
            out[g * (rows // groups):(g + 1) * (rows // groups)] = g
        else:
            out[starts[g]:starts[g + 1]] = g
    return out


def normed(v, kind, eps):
    """(N(v), 1 / sqrt(..)) along the last axis; kind "layer", "rms" or None (v itself)."""
    v = np.asarray(v, dtype=np.float64)
    if kind is None:
        return v, np.ones(v.shape[:-1] + (1,))
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v * r, r


def _rows(v, group, missing, dim):
    """A [groups, dim] vector laid out for the rows (`missing` where there is none or no group)."""
    out = np.full((len(group), dim), missing)
    if v is not None:
        live = group >= 0
        out[live] = np.asarray(v, dtype=np.float64)[group[live]]
    return out


def block_norm(x, norm, eps, weight=None, bias=None, scale=None, shift=None, branch=None, gate=None, post=None,
               post_weight=None, group=None, post_eps=None):
    """(x_out, y); y None where norm is None."""
    x = np.asarray(x, dtype=np.float64)
    T, D = x.shape
    group = np.zeros(T, dtype=np.int64) if group is None else group
    out = x
    if branch is not None:
        h = normed(branch, post, eps if post_eps is None else post_eps)[0]
        h = h if post_weight is None else h * post_weight
        out = x + _rows(gate, group, 1.0, D) * h
    if norm is None:
        return out, None
    y = normed(out, norm, eps)[0]
    y = y if weight is None else y * weight
    y = y if bias is None else y + bias
    return out, y * (1.0 + _rows(scale, group, 0.0, D)) + _rows(shift, group, 0.0, D)


def _through(d, n, r, kind):
    if kind is None:
        return d
    d = d - n * (d * n).mean(-1, keepdims=True) - (d.mean(-1, keepdims=True) if kind == "layer" else 0.0)
    return d * r


def block_norm_backward(dy, dx_out, x_out, norm, eps, weight=None, bias=None, scale=None, shift=None, branch=None,
                        gate=None, post=None, post_weight=None, group=None, post_eps=None, groups=1):
    """The gradients by name, of rows with a group (others are 0)."""
    T, D = np.shape(dx_out if dy is None else dy)
    group = np.zeros(T, dtype=np.int64) if group is None else group
    live = group >= 0
    member = np.zeros((groups, T))
    member[group[live], np.nonzero(live)[0]] = 1.0
    c = np.zeros((T, D)) if dx_out is None else np.array(dx_out, dtype=np.float64)
    out = {}
    if norm is not None:
        n, r = normed(x_out, norm, eps)
        d = np.asarray(dy, dtype=np.float64)
        m = n if weight is None else n * weight
        m = m if bias is None else m + bias
        out["scale"], out["shift"] = member @ (d * m), member @ d
        d = d * (1.0 + _rows(scale, group, 0.0, D))
        out["weight"], out["bias"] = (d * n)[live].sum(0), d[live].sum(0)
        c = c + _through(d if weight is None else d * weight, n, r, norm)
    out["x"] = c
    if branch is not None:
        h, hr = normed(branch, post, eps if post_eps is None else post_eps)
        w = 1.0 if post_weight is None else post_weight
        out["gate"] = member @ (c * h * w)
        d = c * _rows(gate, group, 1.0, D)
        out["post_weight"] = (d * h)[live].sum(0)
        out["branch"] = _through(d * w, h, hr, post)
    return out


def activation(v, act):
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(over="ignore"):
        if act == "silu":
            return v / (1.0 + np.exp(-v))
        if act == "gelu_tanh":  # (1 + tanh u) / 2 = 1 / (1 + e^(-2u)), whose left side cancels far below 0
            return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "gelu":
        return 0.5 * v * np.vectorize(math.erfc, otypes=[np.float64])(-v / math.sqrt(2.0))
    return v


def epilogue(v, bias=None, act="none", gate=None, residual=None, group=None):
    """residual + gate[group] * act(v + bias) for the scaled sums v [M, N]."""
    v = np.asarray(v, dtype=np.float64)
    y = activation(v if bias is None else v + bias, act)
    if gate is not None:
        y = y * _rows(gate, np.zeros(len(y), dtype=np.int64) if group is None else group, 1.0, v.shape[1])
    return y if residual is None else y + residual
