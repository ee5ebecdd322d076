"""GPU parity tests of the token-serving operators where they are long: contexts that a workgroup walks in many tiles,
prompts split over workgroups, batches of hundreds of sequences, wide linears, offsets past 32 bits. Tolerances are
derived in tests/serve_util.py."""
import numpy as np
import pytest
import torch

from oracle import serve
from tests.serve_util import DTYPES, Cache, attention_bounds, f64, gpu, starts, u

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L


def attention(c, cu, q, most, **kw):
    y = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    L.bsq_attention_kv8(q.cuda(), gpu(cu), *c.device(), most, y=y, lse=lse, **kw)
    return y, lse


def check(c, cu, q, y, lse, scale, window=0, full=False):
    ref, rl, parts = serve.attention(f64(q), cu, c.lens, *c.host(), scale, window, full)
    ty, tl = attention_bounds(ref, rl, parts, q.dtype, q.shape[2])
    n = cu[-1]
    got, got_l, empty = f64(y)[:n], f64(lse)[:n], np.isneginf(rl[:n])
    assert np.array_equal(np.isneginf(got_l), empty) and np.all(got[empty] == 0)
    off = np.abs(got - ref[:n]) / ty[:n]
    assert off.max(initial=0.0) <= 1.0, "y off by %.2f bounds at %s" % (off.max(), np.unravel_index(off.argmax(), off.shape))
    with np.errstate(invalid="ignore"):
        assert np.all(empty | (np.abs(got_l - rl[:n]) <= tl[:n]))
    assert torch.all(y[n:] == 7.0) and torch.all(lse[n:] == 7.0)


def queries(seed, T, Hq, D, kind):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((T, Hq, D))).to(DTYPES[kind])


LONG_PROMPTS = [
    # rows, lens, kv heads, q heads, D, page, window, full
    ([40], [3000], 1, 2, 64, 16, 0, False),          # few blocks: split over workgroups
    ([150], [2100], 1, 1, 128, 64, 0, False),
    ([30, 25], [2500, 1300], 2, 4, 128, 32, 0, True),
    ([64], [1700], 1, 2, 256, 256, 0, False),
    ([70], [4000], 1, 2, 64, 16, 1500, False),       # a window that begins inside a tile, far from the start
    ([40, 33], [1600, 2200], 1, 4, 256, 128, 1111, False),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,lens,H,Hq,D,page,window,full", LONG_PROMPTS)
def test_long_prompts(rows, lens, H, Hq, D, page, window, full, kind):
    c, cu, q = Cache(len(lens) + D, lens, H, D, page), starts(rows), queries(D, sum(rows) + 2, Hq, D, kind)
    y, lse = attention(c, cu, q, max(rows), softmax_scale=D ** -0.5, window=window, causal=not full)
    check(c, cu, q, y, lse, D ** -0.5, window, full)


@pytest.mark.parametrize("rows", [[45], [1]])
def test_long_absent_pages(rows):
    """Absent pages throughout a long context, whole tiles of them at its begin and amid it."""
    c, cu, q = Cache(5, [2900], 1, 64, 16), starts(rows), queries(6, rows[0], 4, 64, "bf16")
    c.table[0, :9], c.table[0, 60:75], c.table[0, 100::7], c.table[0, 130] = -1, c.pages, -3, 1 << 30
    y, lse = attention(c, cu, q, rows[0], softmax_scale=0.125)
    check(c, cu, q, y, lse, 0.125)


@pytest.mark.parametrize("rows", [[45], [1]])
def test_long_hidden_nan(rows):
    """NaN codes on absent pages, in front of the window and behind the last token change nothing."""
    c, cu, q = Cache(7, [2400], 1, 128, 64), starts(rows), queries(8, rows[0], 2, 128, "fp16")
    c.table[0, 20] = -1
    want = attention(c, cu, q, rows[0], softmax_scale=0.1, window=1800)
    lo = 2400 - rows[0] - 1800 + 1
    used = np.zeros((c.pages, 64), dtype=bool)
    for t in range(max(lo, 0), 2400):
        if c.table[0, t // 64] >= 0:
            used[c.table[0, t // 64], t % 64] = True
    c.kc[:, 0][~used] = 0x7F
    c.vc[:, 0] = np.where(used[:, None, :], c.vc[:, 0], 0x7F)
    got = attention(c, cu, q, rows[0], softmax_scale=0.1, window=1800)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(c, cu, q, got[0], got[1], 0.1, 1800)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,window", [([1, 1], 0), ([45, 20], 0), ([1, 1], 90), ([45, 20], 90)])
def test_scales_of_pages_that_nobody_sees(rows, window, kind):
    """Pools come uninitialised: scales of pages without tokens, of page 0 among them, and of those in front of the window
    may be anything."""
    lens = [230, 75]
    c, cu, q = Cache(17, lens, 2, 64, 16), starts(rows), queries(18, sum(rows), 4, 64, kind)
    free = next(p for p in range(c.pages) if p not in c.table)
    for a in (c.kc, c.vc, c.ks, c.vs):
        a[[0, free]] = a[[free, 0]]
    at = np.where(c.table == 0, free, np.where(c.table == free, 0, c.table))
    c.table = at.astype(np.int32)
    want = attention(c, cu, q, max(rows), softmax_scale=0.2, window=window)
    check(c, cu, q, *want, 0.2, window)
    seen = [c.table[b, t // 16] for b in range(2) for t in range(lens[b])
            if not window or t > lens[b] - rows[b] - window]
    hidden = np.setdiff1d(np.arange(c.pages), seen)
    assert 0 in hidden and (not window or len(hidden) > 2)
    for bad in (float("nan"), float("inf"), -3e38):
        c.ks[hidden] = c.vs[hidden] = bad
        got = attention(c, cu, q, max(rows), softmax_scale=0.2, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D,H,lens", [(64, 128, [6000, 1, 7100, 5300]), (128, 128, [2300, 4400, 2100]), (256, 64, [3100, 3100, 64, 3700])])
def test_steps_of_many_tiles_a_wave(D, H, lens):
    """So many kv heads that a workgroup takes whole contexts. All heads hold the same codes and queries: the first
    is checked, the others have to be equal to it."""
    c, rows = Cache(D, lens, 1, D, 64), [1] * len(lens)
    q = queries(D + 1, len(lens), 2, D, "bf16")
    dev = [gpu(a) for a in (c.lens, c.table)] + [gpu(a).expand(-1, H, *a.shape[2:]).contiguous() for a in (c.kc, c.vc, c.ks, c.vs)]
    y, lse = L.bsq_attention_kv8(q.cuda().repeat(1, H, 1), gpu(starts(rows)), *dev, 1)
    check(c, starts(rows), q, y[:, :2], lse[:, :2], D ** -0.5)
    assert torch.equal(y, y[:, :2].repeat(1, H, 1)) and torch.equal(lse, lse[:, :2].repeat(1, H))


@pytest.mark.parametrize("most", [1, 2, 30])
def test_hundreds_of_sequences(most):
    """300 sequences of up to `most` rows: the search for a row's sequence, in append and in either attention."""
    rng = np.random.default_rng(most)
    rows = rng.integers(0, most + 1, 300)
    past = rng.integers(0, 90, 300)
    rows[[0, 299]] = 0, most
    cu, lens = starts(rows), list(past + rows)
    c = Cache(most, lens, 1, 64, 16)
    q, k, v = (queries(most + i, int(cu[-1]) + 3, h, 64, "bf16") for i, h in enumerate((4, 1, 1)))
    kc, vc, ks, vs = c.kc.copy(), c.vc.copy(), c.ks.copy(), c.vs.copy()
    serve.append(f64(k), f64(v), cu, c.lens, c.table, kc, vc, ks, vs)
    lens_d, table, gk, gv, gks, gvs = c.device()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), lens_d, table, gk, gv, gks, gvs, q=q.cuda(), q_out=out)
    assert np.array_equal(gk.cpu().numpy(), kc) and np.array_equal(gv.cpu().numpy(), vc)
    assert np.array_equal(f64(gks), ks) and np.array_equal(f64(gvs), vs)
    n = cu[-1]
    assert torch.equal(out[:n].cpu(), q[:n]) and torch.all(out[n:] == 7.0)
    c.kc, c.vc, c.ks, c.vs = kc, vc, ks.astype(np.float32), vs.astype(np.float32)
    y, lse = attention(c, cu, q, most, softmax_scale=0.125)
    check(c, cu, q, y, lse, 0.125)


@pytest.mark.parametrize("rows,most", [([3, 40, 5], 2), ([200, 9], 100), ([5, 6], 4)])
def test_rows_past_the_promised_length(rows, most):
    """Sequences of more rows than max_q_len: the rows up to it are right, the others are not written."""
    lens = [n + 50 for n in rows]
    c, cu, q = Cache(most, lens, 2, 64, 16), starts(rows), queries(3, sum(rows), 4, 64, "bf16")
    y, lse = attention(c, cu, q, most, softmax_scale=0.2)
    ref, rl, parts = serve.attention(f64(q), cu, c.lens, *c.host(), 0.2)
    ty, tl = attention_bounds(ref, rl, parts, q.dtype, 64)
    for b, n in enumerate(rows):
        s, e = cu[b], cu[b] + min(n, most)
        assert np.all(np.abs(f64(y) - ref)[s:e] <= ty[s:e]) and np.all(np.abs(f64(lse) - rl)[s:e] <= tl[s:e])
        assert torch.all((y[e:cu[b + 1]] == 7.0)) and torch.all(lse[e:cu[b + 1]] == 7.0)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_append_rotated_keys_bit_for_bit(kind, interleaved):
    """Half a million rotated keys: every code is that of the key in 64 bits (angles err by some 2^-45 there, so a key
    within that of a border between codes, 2^-4 apart, is not among them)."""
    T, past, H, D = 2000, 37, 2, 128
    c, cu = Cache(21, [past + T], H, D, 64), starts([T])
    k, v = (queries(22 + i, T, H, D, kind) for i in range(2))
    w = L.bsq_rope_inv_freq(D, 500000.0)[0]
    kc, vc, ks, vs = c.kc.copy(), c.vc.copy(), c.ks.copy(), c.vs.copy()
    kr = serve.rope(f64(k), np.arange(past, past + T), f64(w), interleaved, 1.25)
    serve.append(kr, f64(v), cu, c.lens, c.table, kc, vc, ks, vs)
    lens, table, gk, gv, gks, gvs = c.device()
    L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), lens, table, gk, gv, gks, gvs, w.cuda(),
                    L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF, 1.25)
    assert np.array_equal(f64(gks), ks) and np.array_equal(f64(gvs), vs)
    assert np.array_equal(gk.cpu().numpy(), kc) and np.array_equal(gv.cpu().numpy(), vc)


def test_append_many_query_heads_in_place():
    """More query elements than a wave keeps ahead, written over the queries."""
    rows = [3, 1]
    c, cu = Cache(9, [20, 7], 2, 256, 16), starts(rows)
    q, k, v = (queries(10 + i, 6, h, 256, "fp16") for i, h in enumerate((42, 2, 2)))
    w = L.bsq_rope_inv_freq(96, 10000.0)[0].cuda()
    dev = c.device()
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    a = (k.cuda(), v.cuda(), gpu(cu), *dev)
    L.bsq_kv_append(*a, inv_freq=w, q=q.cuda(), q_out=out)
    mine = q.cuda()
    L.bsq_kv_append(*a, inv_freq=w, q=mine, q_out=mine)
    pos = torch.tensor([17, 18, 19, 6], device="cuda")
    assert torch.equal(out[:4], L.bsq_rope(q.cuda()[:4], pos, w))
    assert torch.equal(mine[:4], out[:4]) and torch.equal(mine[4:].cpu(), q[4:])


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K,group,zeros", [
    (1, 40000, 128, 32, True), (2, 17000, 256, 64, False),          # several blocks of rows a wave
    (1, 33, 20480, 128, True), (2, 16, 33280, 64, False),             # more slabs of K than waves
    (3, 6200, 384, 128, True), (16, 6145, 256, 32, False), (20, 6200, 640, 64, True), (40, 6170, 512, 32, True),
    (70, 6200, 256, 128, False)])                                     # two row tiles a wave
def test_wide_int4(M, N, K, group, zeros, kind):
    rng = np.random.default_rng(M + N + K)
    dt = DTYPES[kind]
    x = torch.from_numpy(rng.standard_normal((M, K))).to(dt)
    w = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = torch.from_numpy(rng.uniform(0.001, 0.01, (N, K // group)) * rng.choice([-1, 1], (N, K // group))).to(dt)
    z = rng.integers(8, 16, (N, K // group)).astype(np.uint8) if zeros else None
    ref, size = serve.int4g(f64(x), w, f64(s), z, group)
    y = f64(L.bsq_gemm_int4g(x.cuda(), gpu(w), s.cuda(), None if z is None else gpu(z)))
    terms = (40.0 if kind == "bf16" else 1.0) * size
    bound = u(dt) * np.abs(ref) + (group + K // group + 4) * 2.0 ** -24 * terms + (2.0 ** -25 if kind == "fp16" else 0.0)
    assert np.all(np.abs(y - ref) <= bound), (np.abs(y - ref) / bound).max()


def test_pools_past_4_gib():
    """Pages on both sides of 2^32 bytes of a pool: append and attention do what they do in a small one."""
    H, D, page, many = 8, 256, 256, 8600   # 4.2 GiB each of K and V
    lens, rows = [600, 300], [1, 40]
    small = Cache(11, lens, H, D, page)
    far = np.array([many - 1 - i * 1071 for i in range(small.pages)])   # the last page, and others down to the first
    lens_d, table, gk, gv, gks, gvs = small.device()
    wide = [torch.zeros((many, *t.shape[1:]), dtype=t.dtype, device="cuda") for t in (gk, gv, gks, gvs)]
    at = gpu(far)
    for big, t in zip(wide, (gk, gv, gks, gvs)):
        big[at] = t
    moved = gpu(np.where(small.table >= 0, far[np.clip(small.table, 0, None)], -1).astype(np.int32))
    cu = gpu(starts(rows))
    q, k, v = (queries(12 + i, 41, h, D, "bf16").cuda() for i, h in enumerate((16, H, H)))
    L.bsq_kv_append(k, v, cu, lens_d, table, gk, gv, gks, gvs)
    L.bsq_kv_append(k, v, cu, lens_d, moved, *wide)
    for big, t in zip(wide, (gk, gv, gks, gvs)):
        assert torch.equal(big[at], t)
    for most in (1, 40):
        n = 1 if most == 1 else 41
        c, e = (cu[:2].contiguous(), 1) if most == 1 else (cu, 2)
        want = L.bsq_attention_kv8(q[:n], c, lens_d[:e], table[:e], gk, gv, gks, gvs, most)
        got = L.bsq_attention_kv8(q[:n], c, lens_d[:e], moved[:e], *wide, most)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del wide


def test_rotation_past_2_to_32_elements():
    """Tokens more than 2^32 elements apart."""
    T, H, D, far = 3, 2, 64, (1 << 31) + 64
    base = torch.zeros(2 * far + H * D, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(base, (T, H, D), (far, D, 1))
    vals = queries(13, T, H, D, "bf16").cuda()
    x.copy_(vals)
    pos, w = torch.arange(5, 5 + T, device="cuda"), L.bsq_rope_inv_freq(64, 10000.0)[0].cuda()
    want = L.bsq_rope(vals, pos, w)
    assert torch.equal(L.bsq_rope(x, pos, w), want)
    L.bsq_rope(x, pos, w, y=x)
    assert torch.equal(x, want)
    del base, x


@pytest.mark.parametrize("M", [1, 3])
def test_int4_weights_past_4_gib(M):
    """More than 2^32 bytes of codes: the last rows are what they are alone."""
    N, K, group = (1 << 20) + 1024, 8192, 128
    w = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros((N, K // group), dtype=torch.float16, device="cuda")
    last = torch.randint(0, 256, (512, K // 2), dtype=torch.uint8, device="cuda")
    w[-512:], s[-512:] = last, 0.01
    x = queries(14, M, 1, K, "fp16")[:, 0].cuda()
    y = L.bsq_gemm_int4g(x, w, s)
    ref, size = serve.int4g(f64(x), last.cpu().numpy(), f64(s[-512:]), None, group)
    assert torch.all(y[:, :-512] == 0)
    bound = u(torch.float16) * np.abs(ref) + (group + K // group + 4) * 2.0 ** -24 * size + 2.0 ** -25
    assert np.all(np.abs(f64(y[:, -512:]) - ref) <= bound)
    del w, s


def test_every_operator_on_a_stream_of_its_own():
    """On another stream than the current one each call waits for what that stream holds, and for nothing else."""
    s = torch.cuda.Stream()
    c = Cache(15, [30, 70], 2, 64, 16)
    cu = gpu(starts([1, 1]))
    pos, w = torch.tensor([29, 69], device="cuda"), L.bsq_rope_inv_freq(64, 10000.0)[0].cuda()
    q, k, v = (queries(16 + i, 2, h, 64, "bf16").cuda() for i, h in enumerate((4, 2, 2)))
    codes = gpu(np.random.default_rng(1).integers(0, 256, (32, 128)).astype(np.uint8))
    scale = torch.full((32, 4), 0.01, dtype=torch.bfloat16, device="cuda")

    def run(dev, x):
        out = [L.bsq_rope(x, pos, w), L.bsq_kv_append(k, v, cu, *dev, inv_freq=w, q=x)]
        out += L.bsq_attention_kv8(out[1], cu, *dev, 1)
        return out + [L.bsq_gemm_int4g(out[2].view(2, 256), codes, scale)]

    want = run(c.device(), q)
    dev, late = c.device(), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        for i in range(20):
            big.fill_(i)        # work ahead of the queries' arrival, on this stream
        late.copy_(q)
        got = run(dev, late)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_broadcast_operands_and_no_lse():
    """Queries, keys and values with strides of 0 are what their copies are; lse may be left out."""
    c = Cache(31, [20, 33], 2, 64, 16)
    cu, dev = gpu(starts([3, 2])), c.device()
    one = queries(32, 1, 1, 64, "bf16").cuda()
    wide, shared = one.expand(5, 4, 64), queries(33, 5, 1, 64, "bf16").cuda().expand(5, 2, 64)
    w = L.bsq_rope_inv_freq(64, 10000.0)[0].cuda()
    other = [t.clone() for t in dev]
    q1 = L.bsq_kv_append(shared, shared, cu, *dev, inv_freq=w, q=wide)
    q2 = L.bsq_kv_append(shared.contiguous(), shared.contiguous(), cu, *other, inv_freq=w, q=wide.contiguous())
    assert torch.equal(q1, q2) and all(torch.equal(a, b) for a, b in zip(dev, other))
    y, lse = L.bsq_attention_kv8(wide, cu, *dev, 3)
    y2, lse2 = L.bsq_attention_kv8(wide.contiguous(), cu, *dev, 3)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)
    s = L.Kv8Cache(*(dev[i].data_ptr() for i in (2, 3, 4, 5, 1, 0)), c.pages, 2, 16, 64, 2, dev[1].shape[1], dev[1].shape[1])
    n = L.bsq_attention_kv8_workspace_bytes(2, 5, 3, 4, 2, 64)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    y3 = torch.empty_like(y)
    args = (L.BSQ_BF16, s, cu.data_ptr(), 5, 3, wide.data_ptr(), 0, 0, 4, 0.125, 0, 0, y3.data_ptr(), 256, 64, None)
    assert L.lib.bsq_attention_kv8(*args, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(y3, y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_millions_of_tokens_and_negative_positions(interleaved):
    """More tokens than a dimension of a grid holds, and positions on both sides of 0."""
    T, D = (1 << 23) + 5, 16
    x = torch.randn(T, 1, D, device="cuda").to(torch.bfloat16)
    pos = torch.arange(T, device="cuda") - (1 << 22)
    w = L.bsq_rope_inv_freq(D, 10000.0)[0].cuda()
    layout = L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF
    y = L.bsq_rope(x, pos, w, layout)
    for at in (0, (1 << 22) - 50, T - 200):
        part = slice(at, at + 200)
        assert torch.equal(y[part], L.bsq_rope(x[part], pos[part], w, layout))
        ref = serve.rope(f64(x[part]), pos[part].cpu().numpy(), f64(w), interleaved)
        a = np.abs(f64(x[part]))
        pair = a[..., 0::2] + a[..., 1::2] if interleaved else a[..., :8] + a[..., 8:]
        size = np.repeat(pair, 2, -1) if interleaved else np.concatenate([pair, pair], -1)
        assert np.all(np.abs(f64(y[part]) - ref) <= u(torch.bfloat16) * np.abs(ref) + 2.0 ** -21 * size)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 2, 3, 33])
def test_int4_the_longest_rows(M, kind):
    """K = 2^20."""
    N, K, group = 5, 1 << 20, 128
    rng = np.random.default_rng(M)
    dt = DTYPES[kind]
    x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(dt)
    w = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    s = torch.from_numpy(rng.uniform(0.0001, 0.001, (N, K // group))).to(dt)
    ref, size = serve.int4g(f64(x), w, f64(s), None, group)
    y = f64(L.bsq_gemm_int4g(x.cuda(), gpu(w), s.cuda()))
    # sums over a group, over a wave's groups and over the waves: (group + K / group + 4) roundings at most
    bound = u(dt) * np.abs(ref) + (group + K // group + 4) * 2.0 ** -24 * (40.0 if kind == "bf16" else 1.0) * size + 2.0 ** -25
    assert np.all(np.abs(y - ref) <= bound)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("D,page,window,full", [(64, 16, 0, False), (128, 64, 0, False), (128, 16, 333, False), (256, 256, 0, True)])
def test_prompts_and_steps_in_one_call(D, page, window, full, kind):
    """Chunks of a prompt and single tokens together, with tables wide enough for contexts that a workgroup must not walk
    alone (then either kernel takes its part), and narrow ones."""
    rows, lens = [40, 1, 3, 0, 2, 1, 1], [700, 900, 3, 50, 130, 1, 64]
    c, cu, q = Cache(D + page, lens, 2, D, page), starts(rows), queries(D + 1, sum(rows) + 1, 8, D, kind)
    for width in (c.table.shape[1], (1 << 19) // page):
        table = np.full((len(rows), width), -1, np.int32)
        table[:, :c.table.shape[1]] = c.table
        c.table, narrow = table, c.table
        y, lse = attention(c, cu, q, 40, softmax_scale=D ** -0.5, window=window, causal=not full)
        c.table = narrow
        check(c, cu, q, y, lse, D ** -0.5, window, full)


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, 2200), (256, 0)])
def test_chunks_of_many_heads(D, window):
    """Blocks enough for more than half of the compute units, long enough to be cut in two. All heads hold the same: the
    first is checked, the others have to be equal to it."""
    H, rows, lens = 40, [500], [2600]
    c, q = Cache(D, lens, 1, D, 64), queries(D + 1, 500, 1, D, "bf16")
    dev = [gpu(a) for a in (c.lens, c.table)] + [gpu(a).expand(-1, H, *a.shape[2:]).contiguous() for a in (c.kc, c.vc, c.ks, c.vs)]
    y, lse = L.bsq_attention_kv8(q.cuda().repeat(1, H, 1), gpu(starts(rows)), *dev, 500, window=window)
    check(c, starts(rows), q, y[:, :1], lse[:, :1], D ** -0.5, window)
    assert torch.equal(y, y[:, :1].repeat(1, H, 1)) and torch.equal(lse, lse[:, :1].repeat(1, H))
