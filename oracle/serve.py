"""Oracle of the token-serving operators: rotary positions, the paged E4M3 key/value cache (append
and attention), and linears with 4-bit integer weights and group scales.

TEST INFRASTRUCTURE ONLY (see the package docstring). Plain fp64 NumPy from the definitions in
include/bsq_serve.h, token by token and page by page; inputs are float64 arrays of exactly
representable values.

Pins (``tests/test_oracle_serve.py``): rotations as complex products and by their invariants, the
gradient against differences, frequencies in closed form, a cache worked by hand, attention in
closed form (one token, equal scores) and against an independent two-pass softmax, masks by
perturbing what is hidden, and exact rational sums of the 4-bit product.
"""

import numpy as np

from .codec import E4M3_MAX, e4m3_decode, encode_e4m3


def rope_frequencies(rot, base, scaling="plain", factor=1.0, trained=0, fast=32.0, slow=1.0):
    """fp64 inverse frequencies [rot / 2] and the factor of cosines and sines."""
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    w = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "yarn":
        turns = trained * w / (2 * np.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0.0, 1.0)
        return w * keep + w / factor * (1 - keep), 0.1 * np.log(factor) + 1.0
    return w, 1.0


def rope(x, positions, inv_freq, interleaved=False, factor=1.0, backward=False):
    """x [T, H, D] with its first 2 * len(inv_freq) elements rotated."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    for t, p in enumerate(positions):
        a = float(p) * np.asarray(inv_freq, dtype=np.float64)
        c, s = np.cos(a) * factor, np.sin(a) * factor * (-1.0 if backward else 1.0)
        u, v = x[t, :, first].astype(np.float64), x[t, :, second].astype(np.float64)
        y[t, :, first] = u * c - v * s
        y[t, :, second] = v * c + u * s
    return y


def page_scale(values):
    """The least power of two (>= 2^-126) that brings the largest finite magnitude within E4M3; 0 for zeros."""
    v = np.abs(np.asarray(values, dtype=np.float64))
    a = float(np.max(np.where(np.isfinite(v), v, 0.0), initial=0.0))
    if a == 0.0:
        return 0.0
    e = -126
    while E4M3_MAX * 2.0 ** e < a:
        e += 1
    return 2.0 ** e


def encode(values, scale):
    """E4M3 codes of values / scale: NaN stays NaN, infinities saturate (0 for scale 0)."""
    v = np.asarray(values, dtype=np.float64)
    big = np.finfo(np.float32).max
    ready = np.clip(np.nan_to_num(v, nan=0.0, posinf=big, neginf=-big), -big, big)
    ready = ready / scale if scale > 0 else ready * 0.0
    return np.where(np.isnan(v), np.uint8(0x7F), encode_e4m3(np.clip(ready, -E4M3_MAX, E4M3_MAX)))


def append(k, v, cu, lens, table, k_cache, v_cache, k_scale, v_scale):
    """In place: k, v [T, H, D] (k already rotated) into k_cache [P, H, page, D], v_cache [P, H, D, page] (uint8)."""
    page = k_cache.shape[2]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        past = lens[b] - n
        if n == 0 or past < 0:
            continue
        for j in range(past // page, (lens[b] - 1) // page + 1):
            if j >= table.shape[1] or not 0 <= table[b, j] < k_cache.shape[0]:
                continue
            at = table[b, j]
            lo, hi = max(past, j * page), min(lens[b], (j + 1) * page)
            rows, o0, o1 = slice(cu[b] + lo - past, cu[b] + hi - past), lo - j * page, hi - j * page
            for h in range(k_cache.shape[1]):
                for x, codes, scale in ((k, k_cache[at, h], k_scale), (v, v_cache[at, h].T, v_scale)):
                    before = float(scale[at, h]) if o0 > 0 else 0.0
                    now = max(before, page_scale(x[rows, h]))
                    if o0 > 0 and now != before:
                        codes[:o0] = encode(e4m3_decode(codes[:o0]) * before, now)
                    codes[o0:o1] = encode(x[rows, h], now)
                    scale[at, h] = now


def gather(cache, scale, table_row, tokens, head, transposed):
    """Values [tokens, D] of one head, and whether each token's page is present."""
    page = cache.shape[3] if transposed else cache.shape[2]
    D = cache.shape[2] if transposed else cache.shape[3]
    out, present = np.zeros((tokens, D)), np.zeros(tokens, dtype=bool)
    for j in range((tokens + page - 1) // page):
        if j >= len(table_row) or not 0 <= table_row[j] < cache.shape[0]:
            continue
        lo, hi = j * page, min((j + 1) * page, tokens)
        codes = cache[table_row[j], head]
        codes = codes.T if transposed else codes
        out[lo:hi] = (e4m3_decode(codes) * float(scale[table_row[j], head]))[:hi - lo]
        present[lo:hi] = True
    return out, present


def attention(q, cu, lens, table, k_cache, v_cache, k_scale, v_scale, scale, window=0, full=False):
    """(y [T, Hq, D], lse [T, Hq], parts) with parts: for each row the sums that error bounds need --
    sum_j p_j |v_j| / sum p [T, Hq, D], sum_j |v_j| over the seen tokens / sum p, max_j sum_d |q_d k_jd|, tokens."""
    T, Hq, D = q.shape
    H = k_cache.shape[1]
    y, lse = np.zeros(q.shape), np.full((T, Hq), -np.inf)
    spread, plain, size, count = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, Hq)), np.zeros((T, Hq), dtype=int)
    for b in range(len(lens)):
        n, L = int(cu[b + 1]) - int(cu[b]), max(int(lens[b]), 0)
        for h in range(H if n else 0):
            k, there = gather(k_cache, k_scale, table[b], L, h, False)
            v, _ = gather(v_cache, v_scale, table[b], L, h, True)
            for i in range(n):
                p = L - n + i
                j = np.arange(L)
                seen = there & (np.ones(L, dtype=bool) if full else j <= p) & ((j > p - window) if window else True)
                if not seen.any():
                    continue
                ks, vs = k[seen], v[seen]
                for head in range(h * (Hq // H), (h + 1) * (Hq // H)):
                    s = ks @ q[cu[b] + i, head] * scale
                    m = s.max()
                    e = np.exp(s - m)
                    r = cu[b] + i, head
                    y[r] = e @ vs / e.sum()
                    lse[r] = m + np.log(e.sum())
                    spread[r] = e @ np.abs(vs) / e.sum()
                    plain[r] = np.abs(vs).sum(0) / e.sum()
                    size[r] = (np.abs(ks) @ np.abs(q[r])).max() * abs(scale)
                    count[r] = seen.sum()
    return y, lse, {"spread": spread, "plain": plain, "size": size, "count": count}


def int4g(x, w, scale, zero, group):
    """y [M, N], and sum_k |x| s (c + z) (what its rounding bounds are proportional to)."""
    codes = np.empty((w.shape[0], 2 * w.shape[1]))
    codes[:, 0::2], codes[:, 1::2] = w & 15, w >> 4
    s = np.repeat(np.asarray(scale, dtype=np.float64), group, axis=1)
    z = np.full(codes.shape, 8.0) if zero is None else np.repeat(zero.astype(np.float64), group, axis=1)
    return x @ (s * (codes - z)).T, np.abs(x) @ (np.abs(s) * (codes + z)).T
