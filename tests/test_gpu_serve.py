"""GPU parity tests of the token-serving operators against the fp64 oracle (oracle/serve.py); tolerances are derived
in tests/serve_util.py."""
import numpy as np
import pytest
import torch

from oracle import serve
from oracle.codec import e4m3_decode
from tests.serve_util import DTYPES, Cache, attention_bounds, f64, gpu, starts, u

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L


# ---- rotary positions ---------------------------------------------------------------

def rope_case(T, H, D, rot, kind, interleaved, backward, seed=0, far=100000, factor=1.0):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, H, D))).to(DTYPES[kind])
    pos = rng.integers(0, far, T)
    w, _ = L.bsq_rope_inv_freq(rot, 10000.0)
    return x, pos, w, serve.rope(f64(x), pos, f64(w), interleaved, factor, backward)


def rope_bound(x, ref, rot, factor, kind, interleaved):
    """u |y| + f (|a| + |b|) 2^-21 on rotated elements, the copies exact."""
    m = np.zeros(ref.shape)
    a = np.abs(f64(x))
    first = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    second = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    m[..., first] = m[..., second] = factor * (a[..., first] + a[..., second])
    tiny = 2.0 ** -25 if kind == "fp16" else 0.0   # an fp16 result below the normal range is rounded to 2^-24 steps
    return np.where(m > 0, u(DTYPES[kind]) * np.abs(ref) + m * 2.0 ** -21 + tiny, 0.0)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot,backward", [
    (1, 1, 64, 64, False), (3, 5, 128, 128, True), (70, 8, 128, 64, False), (17, 33, 256, 256, True), (1030, 3, 80, 32, False),
    (5, 2, 7, 6, False), (4, 3, 66, 34, True), (2, 1, 2, 2, False), (9, 40, 1024, 1024, False), (2100, 40, 64, 16, True)])
def test_rope(T, H, D, rot, kind, interleaved, backward):
    factor = 1.25
    x, pos, w, ref = rope_case(T, H, D, rot, kind, interleaved, backward, seed=T, factor=factor)
    y = L.bsq_rope(x.cuda(), gpu(pos), w.cuda(), L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF, factor,
                   backward=backward)
    assert np.all(np.abs(f64(y) - ref) <= rope_bound(x, ref, rot, factor, kind, interleaved))


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_rope_far_positions(kind):
    """Positions to 2^40 and negative ones: the angle is reduced in 64 bits (its product carries 2^-53 of 2^40 turns:
    2^-13 / 2 pi of a turn at most, so the bound grows by 2^-52 p w on each element)."""
    T, H, D = 6, 2, 128
    rng = np.random.default_rng(7)
    x = torch.from_numpy(rng.standard_normal((T, H, D))).to(DTYPES[kind])
    pos = np.array([0, 1, 2 ** 31 + 5, -17, 123456789, 2 ** 40])
    w, _ = L.bsq_rope_inv_freq(D, 10000.0, L.BSQ_ROPE_NTK, 8.0)
    ref = serve.rope(f64(x), pos, f64(w))
    y = f64(L.bsq_rope(x.cuda(), gpu(pos), w.cuda()))
    a = np.abs(f64(x))
    extra = 2.0 ** -51 * np.abs(pos)[:, None, None] * np.tile(f64(w), 2) * (a + np.roll(a, D // 2, -1))
    assert np.all(np.abs(y - ref) <= rope_bound(x, ref, D, 1.0, kind, False) + extra)


def test_rope_strides_and_in_place():
    T, H, D, rot = 37, 6, 128, 128
    x, pos, w, ref = rope_case(T, H, D, rot, "bf16", False, False, seed=11)
    want = L.bsq_rope(x.cuda(), gpu(pos), w.cuda())
    dense = x.cuda()
    assert L.bsq_rope(dense, gpu(pos), w.cuda(), y=dense) is dense and torch.equal(dense, want)
    # a slice of a fused projection, written to a tensor with the heads outermost
    fused = torch.zeros(T, H + 4, D, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:2 + H] = x.cuda()
    out = torch.full((H, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    L.bsq_rope(fused[:, 2:2 + H], gpu(pos), w.cuda(), y=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want)
    # rows off the 16-byte grid, neighbours untouched
    odd = torch.full((T * (H * D + 3) + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(odd, (T, H, D), (H * D + 3, D, 1), 1)
    view.copy_(x)
    L.bsq_rope(view, gpu(pos), w.cuda(), y=view)
    assert torch.equal(view, want)
    gaps = torch.as_strided(odd, (T, 3), (H * D + 3, 1), 1 + H * D)[:-1]
    assert torch.all(gaps == 7.0) and odd[0] == 7.0
    # one head broadcast over all
    y = L.bsq_rope(x.cuda()[:, :1].expand(T, H, D), gpu(pos), w.cuda())
    assert torch.equal(y, want[:, :1].expand(T, H, D))


def test_rope_gradient_against_differences():
    T, H, D, rot = 4, 2, 64, 32
    x, pos, w, _ = rope_case(T, H, D, rot, "fp32", True, False, seed=5)
    dy = torch.from_numpy(np.random.default_rng(6).standard_normal((T, H, D))).float()
    args = gpu(pos), w.cuda(), L.BSQ_ROPE_INTERLEAVED, 1.5
    dx = f64(L.bsq_rope(dy.cuda(), *args, backward=True))
    rng = np.random.default_rng(8)
    for _ in range(20):
        d = torch.from_numpy(rng.standard_normal((T, H, D))).float()
        hi, lo = L.bsq_rope((x + d).cuda(), *args), L.bsq_rope((x - d).cuda(), *args)
        diff = ((f64(hi) - f64(lo)) / 2 * f64(dy)).sum()
        # the map is linear: what differs is the rounding of x +- d (2^-24) and of the rotations (2^-20)
        size = 1.5 * 2 * (np.abs(f64(x)) + np.abs(f64(d))).sum() * np.abs(f64(dy)).max()
        assert abs(diff - (dx * f64(d)).sum()) <= 2.0 ** -19 * size


# ---- append --------------------------------------------------------------------------

def append_case(seed, new, past, H, Hq, D, page, kind, rot, interleaved, extra_rows=0, wild=False):
    rng = np.random.default_rng(seed)
    new, past = np.asarray(new), np.asarray(past)
    c = Cache(seed, list(past + new), H, D, page)
    T = int(new.sum()) + extra_rows
    t = lambda h: torch.from_numpy(rng.standard_normal((T, h, D)) * np.exp(rng.uniform(-4, 4, (T, 1, 1)))).to(DTYPES[kind])  # noqa: E731
    k, v, q = t(H), t(H), t(Hq)
    if wild:
        for x in (k, v):
            x[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0])
    w = L.bsq_rope_inv_freq(rot, 10000.0)[0] if rot else None
    return c, starts(new), k, v, q, w


def expected_append(c, cu, k, v, q, w, past, interleaved, factor):
    pos = np.concatenate([np.arange(p, p + n) for p, n in zip(past, np.diff(cu))] + [[]]).astype(np.int64)
    n = len(pos)
    with np.errstate(invalid="ignore"):
        kr = serve.rope(f64(k)[:n], pos, f64(w), interleaved, factor) if w is not None else f64(k)[:n]
        qr = serve.rope(f64(q)[:n], pos, f64(w), interleaved, factor) if w is not None else f64(q)[:n]
    kc, vc, ks, vs = c.kc.copy(), c.vc.copy(), c.ks.copy(), c.vs.copy()
    serve.append(kr, f64(v), cu, c.lens, c.table, kc, vc, ks, vs)
    return kr, qr, kc, vc, ks, vs


CASES = [
    # new, past, kv heads, q heads, D, page, rot, extra rows
    ([1], [0], 1, 1, 64, 16, 64, 0),
    ([1, 1, 1, 1, 1], [0, 15, 16, 17, 300], 2, 8, 128, 16, 128, 0),
    ([1] * 70, list(range(70)), 1, 4, 64, 32, 32, 3),
    ([0, 40, 0, 1, 7, 0], [5, 3, 0, 63, 64, 9], 2, 6, 128, 64, 64, 5),
    ([130, 260], [0, 61], 3, 3, 128, 128, 0, 0),
    ([300, 5], [200, 255], 1, 2, 256, 256, 256, 1),
    ([33, 64, 65], [31, 0, 1], 2, 2, 256, 32, 128, 0),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,past,H,Hq,D,page,rot,extra", CASES)
def test_append(new, past, H, Hq, D, page, rot, extra, kind, interleaved):
    c, cu, k, v, q, w = append_case(len(new) + D, new, past, H, Hq, D, page, kind, rot, interleaved, extra)
    kr, qr, kc, vc, ks, vs = expected_append(c, cu, k, v, q, w, past, interleaved, 1.25)
    lens, table, gk, gv, gks, gvs = c.device()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    for _ in range(2):  # the second call finds its own tokens there, and changes nothing
        L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), lens, table, gk, gv, gks, gvs, None if w is None else w.cuda(),
                        L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF, 1.25, q.cuda(), out)
        assert np.array_equal(f64(gks), ks) and np.array_equal(f64(gvs), vs)
        assert np.array_equal(gv.cpu().numpy(), vc)
        got = gk.cpu().numpy()
        if rot == 0:
            assert np.array_equal(got, kc)
        else:
            check_keys(c, cu, kr, got, kc, ks, rot, f64(k), interleaved)
        n = cu[-1]
        if rot:
            assert np.all(np.abs(f64(out)[:n] - qr) <= rope_bound(q[:n], qr, rot, 1.25, kind, interleaved))
        else:
            assert torch.equal(out[:n].cpu(), q[:n])
        assert torch.all(out[n:] == 7.0)   # rows of no sequence


def check_keys(c, cu, kr, got, want, ks, rot, k, interleaved):
    """Codes equal the oracle's, except where the rotated key lies within the rotation's error of a border between
    codes: there the value is off by at most the half step 2^-4 (or 2^-10 of the scale) and that error."""
    same = got == want
    page, H = want.shape[2], want.shape[1]
    checked = 0
    for b in range(len(c.lens)):
        n = cu[b + 1] - cu[b]
        for i in range(n):
            t = c.lens[b] - n + i
            at, o = c.table[b, t // page], t % page
            for h in range(H):
                x, s = kr[cu[b] + i, h], ks[at, h]
                a = np.abs(k[cu[b] + i, h])
                m = np.zeros(len(x))
                f = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
                g = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
                m[f] = m[g] = 1.25 * (a[f] + a[g]) * 2.0 ** -21
                err = np.abs(e4m3_decode(got[at, h, o]) * s - x)
                assert np.all(same[at, h, o] | (err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) + m * (1 + 2.0 ** -4)))
                checked += int((~same[at, h, o]).sum())
                same[at, h, o] = True
    assert np.all(same) and checked <= 1e-4 * want.size + 2   # everything else is untouched


def test_append_token_by_token_equals_at_once():
    """Power-of-two scales: pages filled a token at a time hold what they hold when filled at once, up to codes that
    fall below E4M3's normal range on the way (their value is then within half a subnormal step per rescaling)."""
    H, D, page, n = 2, 128, 32, 75
    c, cu, k, v, q, w = append_case(3, [n], [0], H, 2, D, page, "bf16", 64, False)
    one, step = c.device(), c.device()
    L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), *one, w.cuda())
    for i in range(n):
        lens = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        L.bsq_kv_append(k[i:i + 1].cuda(), v[i:i + 1].cuda(), gpu(starts([1])), lens, *step[1:], w.cuda())
    for x, y, sx, sy in ((one[2], step[2], one[4], step[4]), (one[3], step[3], one[5], step[5])):
        assert torch.equal(sx, sy)
        dx, dy = e4m3_decode(x.cpu().numpy()), e4m3_decode(y.cpu().numpy())
        differ = dx != dy
        assert np.all(np.abs(dx - dy)[differ] <= 2.0 ** -8) and np.all(np.abs(dx)[differ] <= 2.0 ** -6)


def test_append_nan_infinities_zeros():
    c, cu, k, v, q, w = append_case(9, [5, 1], [0, 20], 1, 1, 64, 16, "bf16", 0, False, wild=True)
    k[5:], v[5:] = 0.0, 0.0
    c.ks[:], c.vs[:] = 0.25, 0.25
    _, _, kc, vc, ks, vs = expected_append(c, cu, k, v, q, None, [0, 20], False, 1.0)
    lens, table, gk, gv, gks, gvs = c.device()
    L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), lens, table, gk, gv, gks, gvs)
    # NaN codes of either sign stand for NaN
    for got, want in ((gk, kc), (gv, vc)):
        assert np.array_equal(e4m3_decode(got.cpu().numpy()), e4m3_decode(want), equal_nan=True)
    assert np.array_equal(f64(gks), ks) and np.array_equal(f64(gvs), vs)
    allzero = torch.zeros_like(k[:1])
    L.bsq_kv_append(allzero.cuda(), allzero.cuda(), gpu(starts([1, 0])), gpu(np.array([1, 0], np.int32)), table, gk, gv, gks, gvs)
    p = int(c.table[0, 0])
    assert float(gks[p, 0]) == 0.0 and torch.all(gk[p, 0, 0] & 0x7F == 0)


def test_append_skips_what_is_out_of_range():
    """Absent pages, pages past the table, a sequence shorter than its rows: skipped, everything else as ever."""
    new, past = [4, 3, 20, 2], [0, 30, 10, 40]
    c, cu, k, v, q, w = append_case(21, new, past, 2, 2, 64, 16, "bf16", 0, False)
    c.table[0, 0] = -5
    c.table[2, 0] = c.pages            # one past the pool
    c.table = np.ascontiguousarray(c.table[:, :2])   # the last sequence's page (2) is past the table
    c.lens[1] = 2                      # fewer tokens than rows
    _, _, kc, vc, ks, vs = expected_append(c, cu, k, v, q, None, past, False, 1.0)
    lens, table, gk, gv, gks, gvs = c.device()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), lens, table, gk, gv, gks, gvs, q=q.cuda(), q_out=out)
    assert np.array_equal(gk.cpu().numpy(), kc) and np.array_equal(gv.cpu().numpy(), vc)
    assert np.array_equal(f64(gks), ks) and np.array_equal(f64(gvs), vs)
    assert torch.all(out[4:7] == 7.0) and torch.equal(out[7:].cpu(), q[7:]) and torch.equal(out[:4].cpu(), q[:4])


# ---- attention -----------------------------------------------------------------------

def attention_case(seed, rows, lens, H, Hq, D, page, kind, extra=0):
    rng = np.random.default_rng(seed)
    c = Cache(seed, lens, H, D, page)
    T = int(sum(rows)) + extra
    q = torch.from_numpy(rng.standard_normal((T, Hq, D))).to(DTYPES[kind])
    return c, starts(rows), q


def check_attention(c, cu, q, most, scale, window=0, full=False, y=None, lse=None):
    ref, rl, parts = serve.attention(f64(q), cu, c.lens, *c.host(), scale, window, full)
    T = q.shape[0]
    gy = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if y is None else y
    gl = torch.full(q.shape[:2], 7.0, device="cuda") if lse is None else lse
    L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), most, softmax_scale=scale, causal=not full, window=window, y=gy,
                        lse=gl)
    n = cu[-1]
    ty, tl = attention_bounds(ref, rl, parts, q.dtype, q.shape[2])
    ty, tl, ref, rl = ty[:n], tl[:n], ref[:n], rl[:n]
    got, got_l = f64(gy)[:n], f64(gl)[:n]
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(got_l), empty) and np.all(got[empty] == 0)
    off = np.abs(got - ref) / ty
    assert off.max(initial=0.0) <= 1.0, "y off by %.2f bounds at %s" % (off.max(), np.unravel_index(off.argmax(), off.shape))
    with np.errstate(invalid="ignore"):
        assert np.all(empty | (np.abs(got_l - rl) <= tl))
    assert torch.all(gy[n:T] == 7.0) and torch.all(gl[n:T] == 7.0)
    return gy, gl


STEPS = [
    # rows, lens, kv heads, q heads, D, page
    ([1], [1], 1, 1, 64, 16),
    ([1, 1, 1], [1, 16, 17], 2, 8, 128, 16),
    ([1, 0, 1, 1, 1], [63, 50, 64, 65, 129], 2, 10, 128, 32),
    ([1, 1], [777, 300], 2, 2, 256, 64),
    ([1, 1, 1, 1], [5, 0, 2000, 257], 1, 16, 64, 256),
    ([2, 3, 1], [2, 40, 300], 2, 8, 128, 16),
    ([4, 1], [700, 1], 1, 4, 256, 128),
    ([1] * 67, [1 + 13 * i for i in range(67)], 1, 2, 64, 16),
    ([1], [4500], 2, 6, 128, 128),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens,H,Hq,D,page", STEPS)
def test_attention_few_rows(rows, lens, H, Hq, D, page, kind):
    c, cu, q = attention_case(len(lens) + D, rows, lens, H, Hq, D, page, kind, extra=2)
    check_attention(c, cu, q, max(rows), D ** -0.5)


PROMPTS = [
    ([20], [20], 1, 1, 64, 16),
    ([100, 0, 3], [100, 7, 200], 2, 4, 128, 64),
    ([70, 130], [500, 131], 1, 8, 128, 16),
    ([33, 17], [40, 400], 2, 6, 256, 32),
    ([1, 64], [900, 64], 1, 32, 64, 128),
    ([1, 1], [300, 65], 1, 40, 128, 64),
    ([257], [300], 1, 1, 64, 256),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens,H,Hq,D,page", PROMPTS)
def test_attention_many_rows(rows, lens, H, Hq, D, page, kind):
    c, cu, q = attention_case(len(lens) + D + 1, rows, lens, H, Hq, D, page, kind, extra=1)
    check_attention(c, cu, q, max(rows), D ** -0.5)


@pytest.mark.parametrize("window,full", [(1, False), (5, False), (64, False), (100, False), (1 << 40, False), (0, True)])
@pytest.mark.parametrize("rows,lens,H,Hq,D,page", [STEPS[5], STEPS[3], PROMPTS[2], PROMPTS[1]])
def test_attention_masks(rows, lens, H, Hq, D, page, window, full):
    c, cu, q = attention_case(window % 97 + D, rows, lens, H, Hq, D, page, "bf16")
    check_attention(c, cu, q, max(rows), D ** -0.5, window, full)


@pytest.mark.parametrize("rows,lens", [([1, 1, 1], [300, 200, 64]), ([3, 40, 2], [300, 200, 1])])
def test_attention_absent_pages_and_short_sequences(rows, lens):
    """Entries out of the pool, tables narrower than the sequences, sequences shorter than their rows."""
    c, cu, q = attention_case(31, rows, lens, 2, 4, 64, 16, "bf16")
    c.table[0, 3], c.table[0, 0], c.table[1, 2] = -1, c.pages + 3, 1 << 30
    c.table[2, :] = -1
    check_attention(c, cu, q, max(rows), 0.2)
    c.table = np.ascontiguousarray(c.table[:, :5])
    check_attention(c, cu, q, max(rows), 0.2)
    check_attention(c, cu, q, max(rows), 0.2, full=True)
    c.lens[:] = [-7, 0, 2 ** 31 - 1]
    c.table[2, :] = np.arange(5)
    cut = c.lens.copy()
    cut[2] = 80  # what the table has room for; with the causal mask the rows stand far behind it and see all of it
    ref = Cache.__new__(Cache)
    ref.__dict__.update(c.__dict__)
    y, _ = L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), max(rows), softmax_scale=0.2)
    ref.lens = cut
    want, _ = L.bsq_attention_kv8(q.cuda(), gpu(cu), *ref.device(), max(rows), softmax_scale=0.2, causal=False)
    assert torch.equal(y[:cu[2]], torch.zeros_like(y[:cu[2]])) and torch.allclose(y[cu[2]:].float(), want[cu[2]:].float())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens,window", [([1, 1], [70, 200], 0), ([4, 2], [70, 200], 0), ([4, 3], [100, 200], 9),
                                              ([50, 9], [70, 200], 0), ([50, 9], [70, 200], 20)])
def test_attention_hidden_nan(rows, lens, window, kind):
    """NaN codes wherever no row looks, and in tokens that only some rows see: hidden ones change nothing, seen ones make
    exactly the rows that see them NaN, in the element (V) or throughout (K)."""
    H, Hq, D, page = 1, 4, 64, 16
    c, cu, q = attention_case(41, rows, lens, H, Hq, D, page, kind)
    want, want_l = L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), max(rows), softmax_scale=0.2, window=window)
    clean = c.kc.copy(), c.vc.copy()
    used = np.zeros((c.pages, page), dtype=bool)
    for b, n in enumerate(c.lens):
        lo = max(0, n - rows[b] - window + 1) if window else 0
        for t in range(lo, n):
            used[c.table[b, t // page], t % page] = True
    c.kc[:, 0][~used] = 0x7F
    c.vc[:, 0] = np.where(used[:, None, :], c.vc[:, 0], 0xFF)
    y, lse = L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), max(rows), softmax_scale=0.2, window=window)
    assert torch.equal(y, want) and torch.equal(lse, want_l)
    for b in range(2):
        for t in {c.lens[b] - 1, c.lens[b] - rows[b], max(c.lens[b] - rows[b] - 2, 0)}:
            for which in (0, 1):
                c.kc, c.vc = clean[0].copy(), clean[1].copy()
                at, o = c.table[b, t // page], t % page
                if which == 0:
                    c.kc[at, 0, o, 3] = 0x7F
                else:
                    c.vc[at, 0, 37, o] = 0xFF
                y, lse = L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), max(rows), softmax_scale=0.2, window=window)
                bad = torch.zeros(y.shape, dtype=torch.bool)
                for i in range(rows[b]):
                    p = c.lens[b] - rows[b] + i
                    if t <= p and (not window or t > p - window):
                        bad[cu[b] + i, :, :] = which == 0
                        bad[cu[b] + i, :, 37] = True
                assert torch.equal(torch.isnan(y).cpu(), bad)
                assert torch.equal(y.cpu()[~bad], want.cpu()[~bad])


def test_attention_extreme_scores():
    """Scores far apart (one token takes all), a scale of zero (the mean) and a negative one."""
    c, cu, q = attention_case(51, [1, 1], [200, 90], 2, 4, 128, 16, "bf16")
    for scale in (30.0, 0.0, -0.5):
        ref, rl, parts = serve.attention(f64(q), cu, c.lens, *c.host(), scale)
        y, lse = L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), 1, softmax_scale=scale)
        ty, tl = attention_bounds(ref, rl, parts, q.dtype, 128)
        assert np.all(np.abs(f64(lse) - rl) <= tl) and np.all(np.abs(f64(y) - ref) <= ty)


def test_attention_strides():
    """Queries as a slice of a fused projection, the output with the heads outermost, a wide table."""
    c, cu, q = attention_case(61, [1, 30], [100, 70], 2, 4, 64, 16, "fp16")
    lens, table, kc, vc, ks, vs = c.device()
    want, wl = L.bsq_attention_kv8(q.cuda(), gpu(cu), lens, table, kc, vc, ks, vs, 30)
    T = q.shape[0]
    fused = torch.zeros(T, 9, 64, dtype=q.dtype, device="cuda")
    fused[:, 3:7] = q.cuda()
    wide = torch.full((2, table.shape[1] + 5), 3, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out = torch.empty(4, T, 64, dtype=q.dtype, device="cuda")
    y, lse = L.bsq_attention_kv8(fused[:, 3:7], gpu(cu), lens, wide[:, :table.shape[1]], kc, vc, ks, vs, 30,
                                 y=out.transpose(0, 1))
    assert torch.equal(y, want) and torch.equal(lse, wl)


# ---- 4-bit group-scaled linear --------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,group,zeros", [
    (1, 1, 32, 32, True), (1, 17, 128, 128, False), (1, 300, 2048, 64, True), (2, 64, 4096, 128, True), (3, 33, 96, 32, False),
    (4, 40, 2560, 32, True), (7, 50, 1280, 128, True), (16, 100, 640, 64, False), (17, 65, 1024, 32, True), (31, 16, 448, 64, True),
    (33, 130, 512, 128, False), (64, 48, 2176, 128, True), (65, 20, 256, 32, True), (150, 31, 384, 64, False)])
def test_int4(M, N, K, group, zeros, kind):
    rng = np.random.default_rng(M + N + K)
    dt = DTYPES[kind]
    x = torch.from_numpy(rng.standard_normal((M, K))).to(dt)
    w = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = torch.from_numpy(rng.uniform(0.001, 0.01, (N, K // group)) * rng.choice([-1, 1], (N, K // group))).to(dt)
    z = rng.integers(8, 16, (N, K // group)).astype(np.uint8) if zeros else None
    ref, size = serve.int4g(f64(x), w, f64(s), z, group)
    y = f64(L.bsq_gemm_int4g(x.cuda(), gpu(w), s.cuda(), None if z is None else gpu(z)))
    # sums over a group, then over the groups
    terms = (40.0 if kind == "bf16" else 1.0) * size
    bound = u(dt) * np.abs(ref) + (group + K // group + 4) * 2.0 ** -24 * terms + (2.0 ** -25 if kind == "fp16" else 0.0)
    assert np.all(np.abs(y - ref) <= bound), (np.abs(y - ref) / bound).max()


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 2, 5, 40])
def test_int4_small_and_large_values(M, kind):
    """Subnormal activations and scales count, zero points to 255 do, and rows past M and N are left alone."""
    N, K, group = 35, 256, 64
    dt = DTYPES[kind]
    rng = np.random.default_rng(M)
    tiny = 2.0 ** -24 if kind == "fp16" else 2.0 ** -130
    x = torch.from_numpy(rng.integers(-9, 10, (M, K)) * tiny).to(dt)
    w = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    z = rng.integers(8, 256, (N, K // group)).astype(np.uint8)
    s = torch.from_numpy(rng.integers(1, 5, (N, K // group)) * 512.0).to(dt)
    ref, size = serve.int4g(f64(x), w, f64(s), z, group)
    base = torch.full((M + 1, N + 13), 7.0, dtype=dt, device="cuda")
    y = torch.as_strided(base, (M, N), (N + 13, 1))
    L.bsq_gemm_int4g(x.cuda(), gpu(w), s.cuda(), gpu(z), y=y)
    bound = u(dt) * np.abs(ref) + (group + K // group + 4) * 2.0 ** -24 * (40.0 if kind == "bf16" else 1.0) * size + tiny
    assert np.all(np.abs(f64(y) - ref) <= bound)
    assert torch.all(base[:M, N:] == 7.0) and torch.all(base[M] == 7.0)


def test_int4_strided_rows():
    M, N, K = 5, 48, 512
    rng = np.random.default_rng(2)
    wide = torch.from_numpy(rng.standard_normal((M, K + 64))).to(torch.bfloat16).cuda()
    w = gpu(rng.integers(0, 256, (N, K // 2)).astype(np.uint8))
    s = torch.full((N, 4), 0.01, dtype=torch.bfloat16, device="cuda")
    y = L.bsq_gemm_int4g(wide[:, 32:32 + K], w, s)
    assert torch.equal(y, L.bsq_gemm_int4g(wide[:, 32:32 + K].contiguous(), w, s))


# ---- together, as a step of a model uses them ----------------------------------------------

def model_step(p, x, cu, lens, most):
    """Rows of one call: 4-bit projection to q, k, v, positions and append, attention, 4-bit projection back."""
    qkv = L.bsq_gemm_int4g(x, p["w1"], p["s1"], p["z1"], y=p["qkv"][:x.shape[0]]).view(-1, 12, 64)
    L.bsq_kv_append(qkv[:, 8:10], qkv[:, 10:], cu, lens, p["table"], p["kc"], p["vc"], p["ks"], p["vs"], p["freq"],
                    q=qkv[:, :8], q_out=qkv[:, :8])
    y, _ = L.bsq_attention_kv8(qkv[:, :8], cu, lens, p["table"], p["kc"], p["vc"], p["ks"], p["vs"], most,
                               y=p["att"][:x.shape[0]], lse=p["lse"][:x.shape[0]], workspace=p["ws"])
    return L.bsq_gemm_int4g(y.view(-1, 512), p["w2"], p["s2"], y=p["out"][:x.shape[0]])


def model_params(seed, lens, most_rows):
    rng = np.random.default_rng(seed)
    c = Cache(seed, lens, 2, 64, 16)
    _, table, kc, vc, ks, vs = c.device()
    code = lambda n, k: gpu(rng.integers(0, 256, (n, k // 2)).astype(np.uint8))               # noqa: E731
    scale = lambda n, g: gpu(rng.uniform(0.005, 0.01, (n, g))).to(torch.bfloat16)          # noqa: E731
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")                     # noqa: E731
    n = max(L.bsq_attention_kv8_workspace_bytes(len(lens), T, most, 8, 2, 64)
            for T, most in ((most_rows, most_rows), (len(lens), 1)))
    return c, dict(w1=code(768, 256), s1=scale(768, 4), z1=gpu(rng.integers(6, 10, (768, 4)).astype(np.uint8)),
                   w2=code(256, 512), s2=scale(256, 8), table=table, kc=kc, vc=vc, ks=ks, vs=vs,
                   freq=L.bsq_rope_inv_freq(64, 10000.0)[0].cuda(), qkv=e(most_rows, 768), att=e(most_rows, 8, 64),
                   lse=torch.empty(most_rows, 8, device="cuda"), out=e(most_rows, 256),
                   ws=torch.empty(max(n, 256), dtype=torch.uint8, device="cuda"))


def test_prompt_then_steps_equal_the_plain_forms():
    """A prompt and four decode steps of two sequences; each call's attention against the oracle on the cache as it
    stands, each projection and rotation against the oracle on its own input."""
    rng = np.random.default_rng(77)
    total = [40, 23]
    c, p = model_params(77, [t + 4 for t in total], 64)
    lens = np.zeros(2, np.int32)
    for rows in ([40, 23], [1, 1], [1, 1], [1, 1], [1, 1]):
        lens = lens + np.array(rows, np.int32)
        cu = starts(rows)
        x = torch.from_numpy(rng.standard_normal((cu[-1], 256))).to(torch.bfloat16)
        out = model_step(p, x.cuda(), gpu(cu), gpu(lens.astype(np.int32)), max(rows))
        qkv = f64(p["qkv"])[:cu[-1]].reshape(-1, 12, 64)
        ref, size = serve.int4g(f64(x), p["w1"].cpu().numpy(), f64(p["s1"]), p["z1"].cpu().numpy(), 64)
        slack = u(torch.bfloat16) * np.abs(ref) + 72 * 2.0 ** -24 * 40 * size
        ref, slack = ref.reshape(-1, 12, 64), slack.reshape(-1, 12, 64)
        assert np.all(np.abs(qkv - ref)[:, 8:] <= slack[:, 8:])
        y, lse, parts = serve.attention(qkv[:, :8], cu, lens, p["table"].cpu().numpy(), p["kc"].cpu().numpy(),
                                        p["vc"].cpu().numpy(), f64(p["ks"]), f64(p["vs"]), 0.125)
        ty, tl = attention_bounds(y, lse, parts, torch.bfloat16, 64)
        got = f64(p["att"])[:cu[-1]]
        assert np.all(np.abs(got - y) <= ty)
        ref, size = serve.int4g(got.reshape(-1, 512), p["w2"].cpu().numpy(), f64(p["s2"]), None, 64)
        assert np.all(np.abs(f64(out) - ref) <= u(torch.bfloat16) * np.abs(ref) + 76 * 2.0 ** -24 * 40 * size)


def test_captured_step_replays():
    """A decode step captured into a graph, replayed with new lengths and inputs in the same buffers, eager work between;
    a second graph with a workspace of its own alongside."""
    rng = np.random.default_rng(78)
    c, p = model_params(78, [90, 60], 8)
    _, p2 = model_params(78, [90, 60], 8)
    x = torch.empty(2, 256, dtype=torch.bfloat16, device="cuda")
    lens, cu = torch.tensor([50, 20], dtype=torch.int32, device="cuda"), gpu(starts([1, 1]))
    x.copy_(torch.from_numpy(rng.standard_normal((2, 256))))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        model_step(p, x, cu, lens, 1)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model_step(p, x, cu, lens, 1)
    for i in range(5):
        x.copy_(torch.from_numpy(rng.standard_normal((2, 256))))
        lens.add_(torch.tensor([1 + i, 3], dtype=torch.int32, device="cuda"))
        for n in ("kc", "vc", "ks", "vs"):
            p2[n].copy_(p[n])
        graph.replay()
        eager = model_step(p2, x, cu, lens, 1)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        for n in ("kc", "vc", "ks", "vs"):
            assert torch.equal(p[n], p2[n])


def test_two_streams_at_once():
    """Two calls at once, each with a workspace of its own, give what they give alone."""
    cases = [attention_case(91 + i, [1] * 3, [500 + 700 * i, 30, 2000], 2, 8, 128, 32, "bf16") for i in range(2)]
    dev = [(q.cuda(), gpu(cu), c.device()) for c, cu, q in cases]
    alone = [L.bsq_attention_kv8(q, cu, *d, 1)[0].clone() for q, cu, d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    for _ in range(3):
        outs = []
        for s, (q, cu, d) in zip(streams, dev):
            with torch.cuda.stream(s):
                outs.append(L.bsq_attention_kv8(q, cu, *d, 1)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))


def test_same_inputs_give_the_same_bits():
    c, cu, q = attention_case(95, [1] * 5, [3000, 1, 64, 900, 2500], 2, 8, 128, 16, "bf16")
    d = c.device()
    first = L.bsq_attention_kv8(q.cuda(), gpu(cu), *d, 1)
    for _ in range(3):
        again = L.bsq_attention_kv8(q.cuda(), gpu(cu), *d, 1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
