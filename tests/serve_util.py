"""Inputs and tolerances shared by the GPU tests of the token-serving operators.

Tolerances, from the arithmetic (u(t) = eps(t) / 2, the relative error of one rounding to t):
rotation: the angle's rest is rounded to fp32 (2^-25 pi absolute) and sine and cosine carry 2 ulp (2^-22); each
  output is two products and a sum in fp32: |err| <= f (|a| + |b|) 2^-21, then one rounding u(t).
attention, y: the output's rounding u(t) |y|; each probability rounded to t, u(t) sum p|v| / sum p, and below t's
  normal range (fp16) 2^-25 sum |v| / sum p; scores of D products summed in fp32, (D + 4) 2^-24 max sum |q k| scale, which
  moves a probability by that relative amount, in the numerator and in the sum; 2^-20 for exp2 and its argument's
  rounding (arguments below 2^5 in magnitude are compared with scores of that size), and n 2^-24 for the sums over n tokens.
attention, lse: the scores' error, the sum's n 2^-24, 2^-20 for exp2 and log2, 2^-22 of itself.
int4: u(t) |y|; products are exact, and fp32 sums of K terms, taken in any order, err by at most
  K 2^-24 sum |terms|; the terms are x s (c + 128) and x s (z + 128) for bf16, below 40 |x| s (c + z) where c + z >= 8
  (the inputs here), and x s (c - z) for fp16; sums run over a group, then over the groups: (group + K / group + 4) 2^-24.
"""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def u(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def gpu(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


class Cache:
    """A pool of pages with random codes and scales, tables with the pages in random order; entries past a
    sequence's pages hold -1."""

    def __init__(self, seed, lens, heads, dim, page, spare=2, room=0):
        rng = np.random.default_rng(seed)
        pages = [(max(l, 0) + room + page - 1) // page for l in lens]
        self.pages = sum(pages) + spare
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(max(pages, default=1), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        sign = lambda *s: (rng.integers(0, 2, s) << 7).astype(np.uint8)  # noqa: E731
        mag = lambda *s: rng.integers(0, 0x60, s).astype(np.uint8)       # noqa: E731
        P = self.pages
        self.kc, self.vc = mag(P, heads, page, dim) | sign(P, heads, page, dim), mag(P, heads, dim, page) | sign(P, heads, dim, page)
        self.ks = (2.0 ** rng.integers(-5, -1, (P, heads))).astype(np.float32)
        self.vs = (2.0 ** rng.integers(-5, -1, (P, heads))).astype(np.float32)
        self.lens = np.asarray(lens, np.int32)

    def host(self):
        return self.table, self.kc, self.vc, self.ks, self.vs

    def device(self):
        """(seq_lens, table, k_cache, v_cache, k_scale, v_scale), as the binding takes them."""
        return tuple(gpu(a) for a in (self.lens, self.table, self.kc, self.vc, self.ks, self.vs))


def starts(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def attention_bounds(y, lse, parts, dtype, dim):
    n = parts["count"].astype(np.float64)
    score = (dim + 4) * 2.0 ** -24 * parts["size"]
    rel = 2 * (score + 2.0 ** -20 + n * 2.0 ** -24) + u(dtype)
    ty = u(dtype) * np.abs(y) + rel[..., None] * parts["spread"] * 1.01 + 1e-30
    if dtype == torch.float16:
        ty = ty + 2.0 ** -25 * parts["plain"] + 2.0 ** -25   # (the output's own subnormals too)
    tl = score + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return ty, tl
