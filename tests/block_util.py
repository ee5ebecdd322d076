"""Inputs and tolerances shared by the GPU tests of a transformer block's operators.

Tolerances, from the arithmetic (u(t) = eps(t) / 2, the relative error of one rounding to t; all else is fp32, 2^-24 a
step). A row's sums take at most 32 additions in a lane, 6 over the lanes and 8 over the waves, 46 in all, and a few
roundings more: a mean errs by at most 2^-18 of the mean magnitude, a sum of squares by 2^-18 of itself, its root by half.
norms: with e the error of the row that is normed and v = row - mean, N(v) errs by
    r (e + mean e + 2^-18 mean |row| + 2^-23 |row|) + |N| (r rms(e) + 2^-18);
  e is 0 for a loaded row; for x_out it is 2^-22 (|x| + |g h'|) + |g| err(h').
y: |w (1 + s)| err(N) and 2^-22 of each of the terms that are added, then u(t) |y| (fp16: 2^-25 below its normal range).
gradients: c = dx_out + r (d - mean d - N mean(d N)) errs by
    r (2^-18 (|d| + mean |d| + |N| mean |d N|) + err(N) mean |d N| + |N| mean(|d| err(N))) + 2^-18 |r (..)| + 2^-22 |c|,
  and so on through the post norm with the gradient's own error added; a column's sum of T terms, taken over the rows of
  a worker (4, or rows / 1024), then its slots in 32 threads, then those threads, errs by (T / 512 + 64) 2^-24 of the
  terms' magnitudes, and by its terms' errors.
linears: sums of K exact products in fp32, in any order, err by at most K 2^-24 of the terms' magnitudes; the scales 2^-22;
  activations have slopes below 1.2 and err by 2^-15 of themselves and 4e-7 (gelu below -5); then u(bf16).
"""
import numpy as np
import torch

from oracle import block

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def f64(t):
    return t.detach().cpu().double().numpy()


def u(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(y, dtype):
    return u(dtype) * np.abs(y) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def norm_error(row, e, kind, eps):
    """(N, r, bound of N's error) of rows that are themselves off by at most e."""
    n, r = block.normed(row, kind, eps)
    if kind is None:
        return n, r, e + 0.0 * row
    a = np.abs(row)
    mean = (e + 0.0 * row).mean(-1, keepdims=True) + 2.0 ** -18 * a.mean(-1, keepdims=True) if kind == "layer" else 0.0
    rms = np.sqrt(((e + 0.0 * row) ** 2).mean(-1, keepdims=True))
    return n, r, r * (e + mean + 2.0 ** -23 * a) + np.abs(n) * (r * rms + 2.0 ** -18)


def spread(v, group, missing, dim):
    return block._rows(v, group, missing, dim)


def forward_bounds(x, norm, eps, group, weight=None, bias=None, scale=None, shift=None, branch=None, gate=None, post=None,
                   post_weight=None, post_eps=None):
    """(x_out, its bound, y, its bound) before any rounding to the tensors' type."""
    D = x.shape[1]
    out, y = block.block_norm(x, norm, eps, weight, bias, scale, shift, branch, gate, post, post_weight, group, post_eps)
    e = 0.0 * x
    if branch is not None:
        n, _, en = norm_error(branch, 0.0, post, eps if post_eps is None else post_eps)
        w = 1.0 if post_weight is None else np.abs(post_weight)
        g = np.abs(spread(gate, group, 1.0, D)) * w
        e = 2.0 ** -22 * (np.abs(x) + g * np.abs(n)) + g * en
    if norm is None:
        return out, e, None, None
    n, _, en = norm_error(out, e, norm, eps)
    w = 1.0 if weight is None else np.abs(weight)
    b = 0.0 if bias is None else np.abs(bias)
    s = np.abs(1.0 + spread(scale, group, 0.0, D))
    sh = np.abs(spread(shift, group, 0.0, D))
    return out, e, y, s * w * en + 2.0 ** -22 * (s * (w * np.abs(n) + b) + sh)


def backward_bounds(dy, dx_out, x_out, norm, eps, group, groups, weight=None, bias=None, scale=None, shift=None,
                    branch=None, gate=None, post=None, post_weight=None, post_eps=None):
    """({name: gradient}, {name: bound}) before any rounding to the tensors' type."""
    ref = block.block_norm_backward(dy, dx_out, x_out, norm, eps, weight, bias, scale, shift, branch, gate, post,
                                    post_weight, group, post_eps, groups)
    like = dx_out if dy is None else dy
    T, D = like.shape
    live = group >= 0
    member = np.zeros((groups, T))
    member[group[live], np.nonzero(live)[0]] = 1.0
    chain = (T / 512 + 64) * 2.0 ** -24

    def through(d, ed, n, r, en, kind):
        """error of r (d - [mean d] - n mean(d n)) for d off by ed"""
        if kind is None:
            return ed
        m = lambda a: a.mean(-1, keepdims=True)  # noqa: E731
        ad, an = np.abs(d), np.abs(n)
        inner = ad + (m(ad) if kind == "layer" else 0.0) + an * m(ad * an)
        slip = ed + (m(ed) if kind == "layer" else 0.0) + an * m(ed * an) + en * m(ad * an) + an * m(ad * en)
        return r * (2.0 ** -17 * inner + slip)

    tol, c, ec = {}, 0.0 * like if dx_out is None else dx_out, 0.0 * like
    if norm is not None:
        n, r, en = norm_error(x_out, 0.0, norm, eps)
        w = 1.0 if weight is None else weight
        b = 0.0 if bias is None else np.abs(bias)
        ad, an = np.abs(dy), np.abs(n)
        s = 1.0 + spread(scale, group, 0.0, D)
        tol["scale"] = member @ (ad * np.abs(w) * en + (chain + 2.0 ** -21) * ad * (an * np.abs(w) + b))
        tol["shift"] = member @ (chain * ad)
        tol["weight"] = (np.abs(s) * ad * (en + (chain + 2.0 ** -21) * an))[live].sum(0)
        tol["bias"] = ((chain + 2.0 ** -21) * np.abs(s) * ad)[live].sum(0)
        d = dy * s * w
        ec = through(d, 2.0 ** -22 * np.abs(d), n, r, en, norm) + 2.0 ** -22 * np.abs(ref["x"])
        c = ref["x"]
    tol["x"] = ec
    if branch is not None:
        h, hr, eh = norm_error(branch, 0.0, post, eps if post_eps is None else post_eps)
        w = 1.0 if post_weight is None else post_weight
        g = spread(gate, group, 1.0, D)
        term = ec * np.abs(h) + np.abs(c) * eh + (chain + 2.0 ** -21) * np.abs(c * h)
        tol["gate"] = member @ (term * np.abs(w))
        tol["post_weight"] = (np.abs(g) * term)[live].sum(0)
        d = c * g * w
        ed = np.abs(g * w) * ec + 2.0 ** -22 * np.abs(d)
        tol["branch"] = through(d, ed, h, hr, eh, post)
    return ref, tol
