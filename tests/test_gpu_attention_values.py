"""GPU tests of what attention over the E4M3 cache does with the values' range: values that 16 bits do not hold, pages of
scales far apart, pages of zeros, long flat tails, scores past 2^24.

Tolerances, from the arithmetic (u(t) = eps(t) / 2). The second product takes V's codes as they are (exact in fp16) and
weights w = p * (V's page scale) as the sum of two fp16 numbers, in units of a power of two N that the largest weight of the
row is at least half of; weights are at most 2^15 and the largest is above 2^10. The first part is off by less than 2^-10 w
(towards zero), the second by half a step of what is left, so y errs by u(t) |y|; by P_REL w = 2^-10 2^-11 w of each weight,
which for parts below fp16's normal range is 2^-25, at most 2^-35 of the largest weight W, so 2^-35 W sum |code| / sum p;
by the scores, (D + 4) 2^-24 max sum |q k| scale, in numerator and denominator alike; 2^-20 for exp2 and its argument; n
2^-24 for the sums. lse errs by the scores, n 2^-24, 2^-20, and a rounding of N and of the log of the sum, which cancel where
scales of pages are 2^s apart: 2^-23 (|lse| + s); a page of zeros stands at 2^-90.
"""
import numpy as np
import pytest
import torch

from oracle import serve
from oracle.codec import e4m3_decode
from tests.serve_util import DTYPES, Cache, f64, gpu, starts, u

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L

P_REL = 2.0 ** -21   # what two fp16 parts leave of a weight


def queries(seed, T, Hq, D, kind, size=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((T, Hq, D)) * size).to(DTYPES[kind])


def attend(c, cu, q, most, **kw):
    y = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), most, y=y, lse=lse, **kw)
    return y, lse


def reference(c, cu, q, scale, window=0):
    """y, lse in 64 bits, the bounds of both, and which tokens each row sees [rows, tokens] for each sequence."""
    q, (T, Hq, D) = f64(q), q.shape
    H, page = c.kc.shape[1], c.kc.shape[2]
    y, lse, ty, tl, seen_by = np.zeros(q.shape), np.full((T, Hq), -np.inf), np.zeros(q.shape), np.zeros((T, Hq)), []
    for b, n in enumerate(c.lens):
        rows = int(cu[b + 1] - cu[b])
        at = np.arange(n)
        place = n - rows + np.arange(rows)
        seen = at[None] <= place[:, None]
        if window:
            seen &= at[None] > place[:, None] - window
        seen_by.append(seen)
        ids = c.table[b, at // page]
        for h in range(H):
            k = serve.gather(c.kc, c.ks, c.table[b], n, h, False)[0]
            codes = np.stack([e4m3_decode(c.vc[i, h, :, t]) for i, t in zip(ids, at % page)])
            s = c.vs[ids, h].astype(np.float64)
            for i in range(rows):
                m = seen[i]
                for head in range(h * (Hq // H), (h + 1) * (Hq // H)):
                    r = cu[b] + i, head
                    x = k[m] @ q[r] * scale
                    e = np.exp(x - x.max())
                    y[r], lse[r] = (e * s[m]) @ codes[m] / e.sum(), x.max() + np.log(e.sum())
                    score = (D + 4) * 2.0 ** -24 * (np.abs(k[m]) @ np.abs(q[r])).max() * scale
                    rel = 2 * (score + 2.0 ** -20 + m.sum() * 2.0 ** -24) + P_REL
                    w = e * s[m]
                    ty[r] = 1.01 * rel * (w @ np.abs(codes[m])) / e.sum() + 2.0 ** -35 * w.max() * np.abs(codes[m]).sum(0) / e.sum()
                    far = np.ptp(np.log2(s[m][s[m] > 0])) if (s[m] > 0).any() else 0.0
                    tl[r] = score + m.sum() * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * (abs(lse[r]) + far + 90.0 * (s[m] == 0).any())
    return y, lse, ty, tl, seen_by


def check(c, cu, q, y, lse, scale, window=0):
    ref, rl, ty, tl, _ = reference(c, cu, q, scale, window)
    ty = ty + u(q.dtype) * np.abs(ref) + (2.0 ** -25 if q.dtype == torch.float16 else 0.0)   # (fp16 results below 2^-14)
    got, most = f64(y), torch.finfo(q.dtype).max
    big = np.abs(ref) - ty > most
    assert np.array_equal(np.isinf(got) & big, big)
    near = ~big & (np.abs(ref) + ty <= most)
    off, ty = np.abs(got - ref)[near], ty[near]
    assert np.all(off <= ty), "y off by %.2f bounds" % (off / (ty + 1e-300)).max()
    assert np.all(np.abs(f64(lse) - rl) <= tl), (np.abs(f64(lse) - rl) / tl).max()


CASES = [  # rows, lens, window, group: prompts, several rows of a step, one row, windows that begin amid a tile
    ([50], [70], 0, 4), ([4, 3], [70, 130], 0, 4), ([4], [100], 9, 2), ([50, 9], [70, 200], 20, 4), ([1, 2], [150, 64], 0, 8),
    ([150], [2100], 0, 1)]


@pytest.mark.parametrize("kind,top", [("fp16", 2.0 ** 8), ("bf16", 2.0 ** 120)])
@pytest.mark.parametrize("code", [0x78, 0x7E, 0xFE])
@pytest.mark.parametrize("rows,lens,window,group", CASES)
@pytest.mark.parametrize("D", [64, 128])
def test_a_value_past_the_types_range_reaches_only_rows_that_see_it(rows, lens, window, group, kind, top, code, D):
    """One token's value is 65536 and more (2^128 for bf16). Rows that do not see it give the same bits as without it."""
    c, cu, q = Cache(61, lens, 1, D, 16), starts(rows), queries(62, sum(rows), group, D, kind)
    c.vs[:] = top * 2.0 ** -20
    b = len(lens) - 1
    first, last = max(0, lens[b] - rows[b] - window + 1) if window else 0, lens[b] - 1
    for t in {last, first, lens[b] - rows[b], max(first, last - 1)}:
        at, o = c.table[b, t // 16], t % 16
        keep = c.vc[at, 0].copy(), c.vs[at, 0]
        c.vs[at, 0] = top
        c.vc[at, 0] &= 0x87            # the page's other values are small ones
        c.vc[at, 0, 37, o] = 0
        want, want_l = attend(c, cu, q, max(rows), softmax_scale=0.05, window=window)
        c.vc[at, 0, 37, o] = code
        y, lse = attend(c, cu, q, max(rows), softmax_scale=0.05, window=window)
        seen = np.zeros(sum(rows), dtype=bool)
        seen[cu[b]:cu[b + 1]] = reference(c, cu, q, 0.05, window)[4][b][:, t]
        assert seen.any()
        other = torch.from_numpy(~seen)
        assert torch.equal(y.cpu()[other], want.cpu()[other]) and torch.equal(lse, want_l)
        hit = torch.zeros(y.shape, dtype=torch.bool)
        hit[torch.from_numpy(seen), :, 37] = True
        assert torch.equal(y.cpu()[~hit], want.cpu()[~hit]) and not torch.isnan(y).any()
        if kind == "fp16":
            check(c, cu, q, y, lse, 0.05, window)
        c.vc[at, 0], c.vs[at, 0] = keep


@pytest.mark.parametrize("rows", [[3], [40]])
def test_the_largest_fp16_values_through_append(rows):
    """What append makes of 65504 and of infinities (65536 and 114688 in the cache), in the last token."""
    c, cu = Cache(63, [90], 1, 64, 16), starts(rows)
    q, k, v = (queries(64 + i, rows[0], h, 64, "fp16") for i, h in enumerate((4, 1, 1)))
    v[-1, 0, 5], v[-1, 0, 6], v[-1, 0, 7] = 65504.0, -65504.0, float("inf")
    lens, table, kc, vc, ks, vs = c.device()
    L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), lens, table, kc, vc, ks, vs)
    y, lse = L.bsq_attention_kv8(q.cuda(), gpu(cu), lens, table, kc, vc, ks, vs, rows[0], softmax_scale=0.125)
    assert float(vs.max()) == 256.0 and torch.isfinite(y[:-1]).all() and not torch.isnan(y).any()
    c.kc, c.vc, c.ks, c.vs = (t.cpu().numpy() for t in (kc, vc, ks, vs))
    check(c, cu, q, y, lse, 0.125)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens", [([1], [300]), ([40], [300])])
def test_a_large_value_of_no_weight(rows, lens, kind):
    """A token whose probability is 0 in any precision holds 114688: nothing of it arrives, in tiles without masks too."""
    c, cu = Cache(65, lens, 1, 64, 16), starts(rows)
    q = torch.ones(rows[0], 2, 64, dtype=DTYPES[kind])
    c.kc[:] = 0x38                                   # 1.0
    c.ks[:] = 1.0
    at, o = c.table[0, 2], 5
    c.kc[at, 0, o] = 0xB8 + 0x20                     # -16: 1088 below the others
    c.vs[at, 0] = 256.0
    c.vc[at, 0] &= 0x87
    c.vc[at, 0, :, o] = 0x7E
    y, lse = attend(c, cu, q, rows[0], softmax_scale=1.0)
    assert torch.isfinite(y).all()
    check(c, cu, q, y, lse, 1.0)


@pytest.mark.parametrize("kind,lo,hi", [("fp16", -33, 9), ("bf16", -45, 45)])
@pytest.mark.parametrize("rows,lens,window", [([1, 1], [330, 64], 0), ([4], [900], 0), ([40], [300], 0), ([70, 20], [200, 400], 50)])
def test_pages_of_scales_far_apart(rows, lens, window, kind, lo, hi):
    """Every page has a scale of its own, some are 0. Rows that do not see the large pages keep their precision."""
    c, cu, q = Cache(67, lens, 2, 64, 16), starts(rows), queries(68, sum(rows), 4, 64, kind, 0.1)
    rng = np.random.default_rng(69)
    c.vs = (2.0 ** rng.integers(lo, hi, c.vs.shape)).astype(np.float32)
    zero = rng.random(c.vs.shape) < 0.15
    c.vs[zero] = 0.0
    c.vc[zero] = 0
    for b in range(len(lens)):                       # the last pages are the largest: only the last rows see them
        at = c.table[b, (lens[b] - 1) // 16]
        c.vs[at], c.vc[at] = 2.0 ** (hi - 1), c.vc[at] | 1
    y, lse = attend(c, cu, q, max(rows), softmax_scale=0.3, window=window)
    check(c, cu, q, y, lse, 0.3, window)


@pytest.mark.parametrize("rows,lens", [([4], [150]), ([40], [150])])
def test_small_values_and_zeros_below_a_page_that_few_rows_see(rows, lens):
    """Zeros and values of 2^-70 for most rows; the last sees 2^20 as well, which sets the reference of them all."""
    c, cu, q = Cache(79, lens, 1, 64, 16), starts(rows), queries(80, rows[0], 4, 64, "bf16", 0.1)
    c.vs[:] = 2.0 ** -70
    zeros = c.table[0, 1:9:2]
    c.vs[zeros], c.vc[zeros] = 0.0, 0
    c.lens[0] = 145                                  # one token on the last page
    c.vs[c.table[0, 9]] = 2.0 ** 20
    y, lse = attend(c, cu, q, rows[0], softmax_scale=0.3)
    check(c, cu, q, y, lse, 0.3)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens", [([1], [1500]), ([30], [1500])])
def test_contexts_that_begin_with_zeros(rows, lens, kind):
    """More pages of zeros than a wave looks up at once, then small values."""
    c, cu, q = Cache(71, lens, 1, 64, 16), starts(rows), queries(72, rows[0], 4, 64, kind, 0.1)
    zeros = c.table[0, :80]
    c.vs[zeros], c.vc[zeros] = 0.0, 0
    c.vs[c.table[0, 80:]] = 2.0 ** -20
    y, lse = attend(c, cu, q, rows[0], softmax_scale=0.3)
    check(c, cu, q, y, lse, 0.3)
    c.vs[:], c.vc[:] = 0.0, 0                        # and nothing else
    y, lse = attend(c, cu, q, rows[0], softmax_scale=0.3)
    assert torch.all(y == 0)
    check(c, cu, q, y, lse, 0.3)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 17])
@pytest.mark.parametrize("below", [9.0, 17.375])
def test_one_strong_token_over_a_long_flat_tail(rows, below, kind):
    """20 000 tokens `below` nats under one: together they hold 0.06 % to 71 % of the sum, and as much of y. So many kv
    heads that a workgroup walks a long part of the context."""
    n, H = 20_000, 128
    c, cu = Cache(73, [n], 1, 64, 256), starts([rows])
    c.kc[:], c.ks[:], c.vc[:], c.vs[:] = 0, 1.0, 0x38, 1.0
    at = c.table[0, 3]
    c.kc[at, 0, 9], c.vc[at, 0, :, 9] = 0x38, 0       # the strong one: score 64 * scale, value 0
    dev = [gpu(a) for a in (c.lens, c.table)] + [gpu(a).expand(-1, H, *a.shape[2:]).contiguous() for a in (c.kc, c.vc, c.ks, c.vs)]
    q = torch.ones(rows, H, 64, dtype=DTYPES[kind], device="cuda")
    y, lse = L.bsq_attention_kv8(q, gpu(cu), *dev, rows, softmax_scale=below / 64)
    for i in range(rows):
        tail = (n - rows + i) * np.exp(-below)
        ref = tail / (1 + tail)
        # weights' roundings and the flat floor 2^-35 of each, sums, scores of one product exact
        bound = u(q.dtype) * ref + (P_REL + 2 * (2.0 ** -20 + n * 2.0 ** -24)) * ref + 2.0 ** -35 * n / (1 + tail) + \
            68 * 2.0 ** -24 * below * ref + (2.0 ** -25 if kind == "fp16" else 0.0)
        assert np.all(np.abs(f64(y[i]) - ref) <= bound), (f64(y[i]).min(), ref, bound)
        assert np.all(np.abs(f64(lse[i]) - (below + np.log1p(tail))) <= n * 2.0 ** -24 + 68 * 2.0 ** -24 * below + 2.0 ** -20 + 2.0 ** -22 * below)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [1, 20])
def test_scores_past_2_to_24(rows, kind):
    """Scores of 1e9, where a step of fp32 is 64: equal ones share equally among pages of one scale, one far above the
    others takes all whatever the scales, and nothing becomes NaN."""
    lens = [200]
    c, cu = Cache(75, lens, 1, 64, 16), starts([rows])
    q = torch.ones(rows, 2, 64, dtype=DTYPES[kind])
    c.kc[:], c.ks[:] = 0x38, 1.0
    for scale in (1e9 / 64, -1e9 / 64):
        c.vs[:] = 0.5
        y, lse = attend(c, cu, q, rows, softmax_scale=scale)
        v = serve.gather(c.vc, c.vs, c.table[0], 200, 0, True)[0]
        for i in range(rows):
            seen = v[:200 - rows + 1 + i]
            err = (u(q.dtype) + P_REL + 2.0 ** -15) * np.abs(seen).mean(0) + 2.0 ** -25
            assert np.all(np.abs(f64(y[i]) - seen.mean(0)) <= err)
        assert np.all(np.abs(f64(lse) - scale * 64) <= 2.0 ** -20 * 1e9)
    c.vs[c.table[0, ::2]] = 2.0 ** 7
    y, _ = attend(c, cu, q, rows, softmax_scale=1e9 / 64)
    assert torch.isfinite(y).all()
    at = c.table[0, 4]
    c.kc[at, 0, 3] = 0x40                            # 2.0: 1e9 above the others
    y, lse = attend(c, cu, q, rows, softmax_scale=1e9 / 64)
    want = serve.gather(c.vc, c.vs, c.table[0], 200, 0, True)[0][67]
    assert np.all(np.abs(f64(y) - want) <= u(q.dtype) * np.abs(want) + P_REL * np.abs(want))
    assert np.all(np.abs(f64(lse) - 2e9) <= 2.0 ** -20 * 2e9)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens,D", [([1, 1], [700, 33], 128), ([3], [500], 64), ([1], [600], 256), ([60], [600], 64), ([40], [500], 128),
                                         ([20], [300], 256)])
def test_weights_in_as_many_bits_as_their_sum(rows, lens, D, kind):
    """Scores near 1, values of either sign that cancel for the most part: y's own rounding is far below sum p |v|, of which
    weights in 11 bits would cost 2^-12 here and there."""
    c, cu, q = Cache(77, lens, 1, D, 16), starts(rows), queries(78, sum(rows), 4, D, kind, 0.05)
    c.vs[:] = 0.5
    y, lse = attend(c, cu, q, max(rows), softmax_scale=D ** -0.5)
    check(c, cu, q, y, lse, D ** -0.5)
