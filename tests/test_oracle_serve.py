"""Pins of the token-serving oracle (oracle/serve.py)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import serve
from oracle.codec import e4m3_decode


def test_frequencies_in_closed_form():
    w, f = serve.rope_frequencies(8, 10000.0)
    assert f == 1.0 and np.allclose(w, [1.0, 0.1, 0.01, 0.001], rtol=1e-15)
    assert np.allclose(serve.rope_frequencies(8, 10000.0, "linear", 4.0)[0], w / 4, rtol=1e-15)
    # NTK: the first pair keeps its frequency, the last is stretched by the whole factor
    n = serve.rope_frequencies(8, 10000.0, "ntk", 4.0)[0]
    assert n[0] == 1.0 and np.isclose(n[-1], w[-1] / 4, rtol=1e-14)
    # YaRN: pairs of more than `fast` turns over the trained length are kept, of fewer than `slow` stretched
    y, f = serve.rope_frequencies(8, 10000.0, "yarn", 4.0, trained=1000)
    assert y[0] == w[0] and np.isclose(y[3], w[3] / 4, rtol=1e-15) and w[1] / 4 < y[1] < w[1]
    assert np.isclose(f, 0.1 * np.log(4.0) + 1, rtol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 10))
    w = np.array([1.0, 0.3, 0.07])
    pos = np.array([0, 5, 1000])
    y = serve.rope(x, pos, w, interleaved, factor=1.25)
    turn = 1.25 * np.exp(1j * pos[:, None, None] * w)
    z = (x[..., 0:6:2] + 1j * x[..., 1:6:2]) if interleaved else (x[..., :3] + 1j * x[..., 3:6])
    z = z * turn
    got = (y[..., 0:6:2] + 1j * y[..., 1:6:2]) if interleaved else (y[..., :3] + 1j * y[..., 3:6])
    assert np.allclose(got, z, rtol=0, atol=1e-14) and np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(y[0, :, :6], 1.25 * x[0, :, :6])            # position 0
    back = serve.rope(serve.rope(x, pos, w, interleaved), pos, w, interleaved, backward=True)
    assert np.allclose(back, x, rtol=0, atol=1e-14)                # the transpose is the inverse


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_gradient_against_differences(interleaved):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 1, 6)), rng.standard_normal((2, 1, 6))
    w, pos = np.array([0.7, 0.2]), np.array([3, 11])
    dx = serve.rope(dy, pos, w, interleaved, factor=1.1, backward=True)
    dx[..., 4:] = dy[..., 4:]
    for i in np.ndindex(x.shape):
        e = np.zeros(x.shape)
        e[i] = 0.5
        hi = (serve.rope(x + e, pos, w, interleaved, 1.1) * dy).sum()
        lo = (serve.rope(x - e, pos, w, interleaved, 1.1) * dy).sum()
        assert abs((hi - lo) - dx[i]) < 1e-12


def test_page_scale():
    assert serve.page_scale([0.0, -0.0]) == 0.0
    assert serve.page_scale([448.0]) == 1.0 and serve.page_scale([np.nextafter(448.0, 500)]) == 2.0
    assert serve.page_scale([224.0, -3.0]) == 0.5 and serve.page_scale([np.nan, np.inf, 1.0]) == 2.0 ** -8
    assert serve.page_scale([1e-44]) == 2.0 ** -126


def test_append_by_hand():
    """One head, D 2, pages of 2 tokens: scales and codes worked by hand."""
    kc, vc = np.full((3, 1, 2, 2), 0x55, np.uint8), np.full((3, 1, 2, 2), 0x55, np.uint8)
    ks, vs = np.full((3, 1), 7.0, np.float32), np.full((3, 1), 7.0, np.float32)
    table = np.array([[2, 0]])
    k = np.array([[[448.0, 1.0]]])
    v = np.array([[[0.0, 0.0]]])
    serve.append(k, v, [0, 1], [1], table, kc, vc, ks, vs)
    assert ks[2, 0] == 1.0 and vs[2, 0] == 0.0                      # a first token starts the page anew
    assert np.array_equal(e4m3_decode(kc[2, 0, 0]), [448.0, 1.0]) and np.all(kc[2, 0, 1] == 0x55)
    assert np.array_equal(vc[2, 0, :, 0], [0, 0]) and np.all(vc[2, 0, :, 1] == 0x55)
    # the second token is larger: the scale grows fourfold, the first token's codes follow
    serve.append(np.array([[[1500.0, -4.0]]]), np.array([[[2.0, -1.0]]]), [0, 1], [2], table, kc, vc, ks, vs)
    assert ks[2, 0] == 4.0 and vs[2, 0] == 2.0 ** -7
    assert np.array_equal(e4m3_decode(kc[2, 0, 0]), [112.0, 0.25])
    assert np.array_equal(e4m3_decode(kc[2, 0, 1]), [384.0, -1.0])   # 375 -> 384 (steps of 32: 352, 384)
    assert np.array_equal(e4m3_decode(vc[2, 0]), [[0.0, 256.0], [0.0, -128.0]])
    assert np.all(kc[0] == 0x55) and np.all(kc[1] == 0x55)
    # a third token opens page 0; appending again changes nothing
    for _ in range(2):
        serve.append(np.array([[[3.0, 0.0]]]), v, [0, 1], [3], table, kc, vc, ks, vs)
        assert ks[0, 0] == 2.0 ** -7 and e4m3_decode(kc[0, 0, 0, 0]) == 384.0 and np.all(kc[0, 0, 1] == 0x55)


def test_append_nan_and_infinities():
    kc, vc = np.zeros((1, 1, 4, 2), np.uint8), np.zeros((1, 1, 2, 4), np.uint8)
    ks, vs = np.zeros((1, 1), np.float32), np.zeros((1, 1), np.float32)
    k = np.array([[[np.nan, 1.0]], [[np.inf, -np.inf]]])
    serve.append(k, k, [0, 2], [2], np.array([[0]]), kc, vc, ks, vs)
    assert ks[0, 0] == 2.0 ** -8
    assert np.isnan(e4m3_decode(kc[0, 0, 0, 0])) and np.array_equal(e4m3_decode(kc[0, 0, 1]), [448.0, -448.0])


def _cache(rng, B, page, lens, H, D, spare=1):
    pages = [(l + page - 1) // page for l in lens]
    P = sum(pages) + spare
    order = rng.permutation(P)
    table, at = np.full((B, max(max(pages), 1)), -1), 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    codes = lambda *s: rng.integers(0, 0x70, s).astype(np.uint8) | (rng.integers(0, 2, s).astype(np.uint8) << 7)  # noqa: E731
    return (table, codes(P, H, page, D), codes(P, H, D, page),
            2.0 ** rng.integers(-7, -4, (P, H)).astype(np.float64), 2.0 ** rng.integers(-7, -4, (P, H)).astype(np.float64))


def test_attention_closed_forms_and_two_pass():
    rng = np.random.default_rng(3)
    lens, cu = [1, 37, 0], [0, 1, 4, 4]
    table, kc, vc, ks, vs = _cache(rng, 3, 16, lens, 2, 4)
    q = rng.standard_normal((4, 4, 4))
    y, lse, _ = serve.attention(q, cu, lens, table, kc, vc, ks, vs, 0.5)
    v0, _ = serve.gather(vc, vs, table[0], 1, 0, True)
    k0, _ = serve.gather(kc, ks, table[0], 1, 0, False)
    assert np.allclose(y[0, 0], v0[0], rtol=1e-14)                 # one token: its value and score
    assert np.isclose(lse[0, 1], 0.5 * (k0[0] @ q[0, 1]), rtol=1e-13)
    k, _ = serve.gather(kc, ks, table[1], 37, 1, False)
    v, _ = serve.gather(vc, vs, table[1], 37, 1, True)
    for i in range(3):                                             # rows 1..3 at positions 34..36
        w = np.exp(0.5 * k[:35 + i] @ q[1 + i, 2])
        assert np.allclose(y[1 + i, 2], (w[:, None] * v[:35 + i]).sum(0) / w.sum(), rtol=1e-12)
        assert np.isclose(lse[1 + i, 2], np.log(w.sum()), rtol=1e-12)
    z, zl, _ = serve.attention(np.zeros_like(q), cu, lens, table, kc, vc, ks, vs, 0.5)
    assert np.allclose(z[3, 3], v[:37].mean(0), rtol=1e-12) and np.isclose(zl[3, 3], np.log(37))  # equal scores


def test_attention_masks_by_perturbation():
    """What is hidden may be anything; what is seen matters."""
    rng = np.random.default_rng(4)
    lens, cu = [50], [0, 3]
    table, kc, vc, ks, vs = _cache(rng, 1, 16, lens, 1, 4)
    q = rng.standard_normal((3, 1, 4))
    for window, full in ((0, False), (5, False), (0, True)):
        base = serve.attention(q, cu, lens, table, kc, vc, ks, vs, 0.3, window, full)[0]
        for j in range(64):
            if j // 16 >= table.shape[1]:
                continue
            k2, v2 = kc.copy(), vc.copy()
            k2[table[0, j // 16], 0, j % 16] = 0x7F
            v2[table[0, j // 16], 0, :, j % 16] = 0x7F
            got = serve.attention(q, cu, lens, table, k2, v2, ks, vs, 0.3, window, full)[0]
            for i in range(3):
                p = 47 + i
                sees = j < 50 and (full or j <= p) and (not window or j > p - window)
                assert np.array_equal(got[i], base[i]) != sees, (window, full, j, i)
    # rows before the sequence's start, and a missing page
    y, lse, _ = serve.attention(q, cu, [1], table, kc, vc, ks, vs, 0.3)
    assert np.all(y[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.isfinite(lse[2, 0])
    gone = table.copy()
    gone[0, 1] = -1
    assert np.array_equal(serve.gather(kc, ks, gone[0], 50, 0, False)[1], (np.arange(50) // 16) != 1)


def test_int4g_exact():
    rng = np.random.default_rng(5)
    x = rng.integers(-8, 9, (3, 64)) / 8.0
    w = rng.integers(0, 256, (5, 32)).astype(np.uint8)
    s = rng.integers(1, 9, (5, 2)) / 16.0
    z = rng.integers(0, 16, (5, 2)).astype(np.uint8)
    for zero in (z, None):
        y, _ = serve.int4g(x, w, s, zero, 32)
        for m in range(3):
            for n in range(5):
                ref = Fraction(0)
                for k in range(64):
                    c = int(w[n, k // 2] >> (4 * (k % 2))) & 15
                    ref += Fraction(x[m, k]) * Fraction(s[n, k // 32]) * (c - (8 if zero is None else int(z[n, k // 32])))
                assert Fraction(y[m, n]) == ref
