"""GPU parity tests of the gated residual with its norms, and of its gradient, against the fp64 oracle (oracle/block.py);
tolerances are derived in tests/block_util.py."""
import numpy as np
import pytest
import torch

from oracle import block
from oracle.codec import e2m1_decode, e4m3_decode
from tests.block_util import DTYPES, backward_bounds, f64, forward_bounds, rounded

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L

KINDS = {None: 0, "layer": 1, "rms": 2}
EPS, POST_EPS = 1e-6, 1e-3


def vectors(seed, T, D, kind, groups=1, strided=False, **want):
    """Inputs on the GPU by name; `want` says which. strided: modulation vectors are slices of one tensor."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, size=1.0, mean=0.0: (torch.randn(*s, generator=g, dtype=torch.float64) * size + mean).to(DTYPES[kind])  # noqa: E731
    v = {"x": n(T, D, size=2.0, mean=0.7)}
    mod = n(groups, 3 * D + 8 * (not strided), size=0.6).cuda()
    for i, k in enumerate(("scale", "shift", "gate")):
        m = mod[:, i * D:(i + 1) * D]
        v[k] = (m if strided else m.contiguous()) if want.get(k) else None
    v["branch"] = n(T, D, size=1.5, mean=-0.2) if want.get("branch") else None
    v["weight"] = n(D, size=0.4, mean=1.0) if want.get("weight") else None
    v["bias"] = n(D, size=0.4) if want.get("bias") else None
    v["post_weight"] = n(D, size=0.4, mean=0.8) if want.get("post_weight") else None
    return {k: None if t is None else t.cuda() for k, t in v.items()}


def doubles(v):
    return {k: None if t is None else f64(t) for k, t in v.items()}


ALL = dict(scale=1, shift=1, gate=1, branch=1, weight=1, bias=1, post_weight=1)
# rows, dim, norm, post, groups, starts, vectors
CASES = [
    (1, 8, "rms", None, 1, None, {}),
    (1, 64, "layer", None, 1, None, dict(scale=1, shift=1)),
    (5, 72, "layer", "rms", 3, [0, 0, 3, 5], ALL),
    (9, 512, "rms", "layer", 4, [0, 2, 2, 7, 8], ALL),
    (66, 520, "rms", None, 2, None, dict(branch=1, gate=1, scale=1)),
    (130, 1024, "layer", None, 1, None, dict(branch=1, weight=1, bias=1)),
    (37, 1032, "layer", "rms", 1, None, dict(branch=1, weight=1, post_weight=1)),
    (301, 2048, "rms", "rms", 70, list(range(0, 70)) + [290], ALL),
    (24, 2560, "layer", None, 24, None, dict(branch=1, gate=1, scale=1, shift=1)),
    (3, 4096, "rms", "rms", 1, None, dict(branch=1, weight=1, post_weight=1)),
    (17, 5120, "layer", None, 2, [0, 9, 17], dict(branch=1, gate=1, scale=1, shift=1)),
    (4, 6152, "rms", "layer", 1, None, dict(branch=1)),
    (6, 8192, "layer", "layer", 2, None, ALL),
    (3, 12288, "rms", None, 1, None, dict(weight=1)),
    (4, 16384, "layer", "rms", 2, None, ALL),
    (1030, 128, "layer", None, 5, [0, 1, 500, 500, 800, 1000], dict(branch=1, gate=1, scale=1, shift=1)),
]


def groups_of(T, groups, starts):
    return block.group_of_rows(T, groups, starts), None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda()


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,D,norm,post,groups,starts,want", CASES)
def test_forward(T, D, norm, post, groups, starts, want, kind):
    v = vectors(T + D, T, D, kind, groups, strided=T % 2 == 1, **want)
    group, st = groups_of(T, groups, starts)
    if not any(want.get(k) for k in ("scale", "shift", "gate")):
        group = np.zeros(T, dtype=np.int64)
    out, eo, y, ey = forward_bounds(norm=norm, eps=EPS, post=post, post_eps=POST_EPS, group=group, **doubles(v))
    y_buf = torch.full((T, D), 7.0, dtype=DTYPES[kind], device="cuda")
    x_buf = torch.full((T, D), 7.0, dtype=DTYPES[kind], device="cuda") if want.get("branch") else None
    got, scale, x_out = L.bsq_block_norm(norm=KINDS[norm], eps=EPS, post=KINDS[post], post_eps=POST_EPS, starts=st,
                                         y=y_buf, x_out=x_buf, **v)
    assert got is y_buf and x_out is x_buf and scale is None
    live = group >= 0
    assert np.all(np.abs(f64(got) - y)[live] <= (ey + rounded(y, DTYPES[kind]))[live])
    assert np.all(f64(got)[~live] == 7.0)
    if x_buf is not None:
        assert np.all(np.abs(f64(x_out) - out)[live] <= (eo + rounded(out, DTYPES[kind]))[live])
        assert np.all(f64(x_out)[~live] == 7.0)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D,norm,post,groups,starts,want", [c for c in CASES if c[1] % 32 == 0])
def test_forward_encoded(T, D, norm, post, groups, starts, want, kind):
    v = vectors(T + D + 1, T, D, kind, groups, **want)
    group, st = groups_of(T, groups, starts)
    if not any(want.get(k) for k in ("scale", "shift", "gate")):
        group = np.zeros(T, dtype=np.int64)
    out, eo, y, ey = forward_bounds(norm=norm, eps=EPS, post=post, post_eps=POST_EPS, group=group, **doubles(v))
    live = group >= 0
    args = dict(norm=KINDS[norm], eps=EPS, post=KINDS[post], post_eps=POST_EPS, starts=st, **v)
    q, d, x_out = L.bsq_block_norm(out_format=L.BSQ_FMT_FP8R, **args)
    d = f64(d)[live]
    # the scale: the largest |y| (off by its error) / 448, rounded once
    most = np.abs(y)[live].max(-1)
    assert np.all(np.abs(d - most / 448) <= ey[live].max(-1) / 448 + 2.0 ** -22 * d)
    # the codes: half a step of E4M3 (2^-4 of the value, 2^-10 below its normal range) on y / d, whose reciprocal and
    # product round twice
    v8 = e4m3_decode(q.cpu().numpy()).astype(np.float64)[live] * d[:, None]
    assert np.all(np.abs(v8 - y[live]) <= (2.0 ** -4 + 2.0 ** -20) * np.abs(y[live]) + 2.0 ** -10 * d[:, None]
                  + 1.1 * ey[live] + 1.1 * ey[live].max(-1, keepdims=True))
    g = np.float32(np.abs(y[live]).max() / (6 * 448) * 1.01)
    q, s, _ = L.bsq_block_norm(out_format=L.BSQ_FMT_NVFP4, y_global=torch.tensor([g], device="cuda"), **args)
    g = float(g)
    s = e4m3_decode(s.cpu().numpy()).astype(np.float64)[live]
    by = np.abs(y[live]).reshape(len(s), -1, 16)
    want_s, es = by.max(-1) / 6 / g, ey[live].reshape(by.shape).max(-1) / 6 / g
    assert np.all(np.abs(s - want_s) <= (2.0 ** -4 + 2.0 ** -20) * want_s + 2.0 ** -10 + 1.1 * es)
    # the codes: half a step of E2M1 (1/4 up to 2, then a quarter of the value at most; values up to 6 (1 + 2^-4) saturate)
    code = q.cpu().numpy()[live]
    v4 = np.stack([e2m1_decode(code & 15), e2m1_decode(code >> 4)], -1).reshape(len(code), -1, 16).astype(np.float64)
    unit = s[..., None] * g
    yb = y[live].reshape(by.shape)
    tiny = s[..., None] * 0 + (s[..., None] == 0) * 2.0 ** -9 * g * 6   # a block whose scale falls to 0 is lost
    assert np.all(np.abs(v4 * unit - yb) <= np.maximum(0.25 * unit, np.abs(yb) / 4) * (1 + 2.0 ** -20)
                  + 2.0 ** -10 * 6 * g + tiny + 1.1 * ey[live].reshape(by.shape))


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,D,norm,post,groups,starts,want", CASES + [
    (420, 1536, "rms", "layer", 6, None, ALL),
    (700, 4096, "layer", None, 3, [0, 200, 201, 690], dict(branch=1, gate=1, scale=1, shift=1)),
    (9, 64, None, "rms", 2, [0, 4, 8], dict(branch=1, gate=1, post_weight=1)),
    (40, 2560, None, None, 2, None, dict(branch=1, gate=1)),
    (5000, 64, "rms", "rms", 2, [0, 4999, 5000], ALL), (2000, 4096, "layer", None, 1, None, dict(weight=1, bias=1)),
    (700, 4608, "layer", "rms", 7, None, ALL)])
def test_backward(T, D, norm, post, groups, starts, want, kind):
    v = vectors(T + D + 2, T, D, kind, groups, strided=T % 2 == 0, **want)
    group, st = groups_of(T, groups, starts)
    if not any(want.get(k) for k in ("scale", "shift", "gate")):
        group = np.zeros(T, dtype=np.int64)
    g = torch.Generator().manual_seed(T)
    dy = torch.randn(T, D, generator=g).to(DTYPES[kind]).cuda() if norm else None
    do = torch.randn(T, D, generator=g).to(DTYPES[kind]).cuda() if want.get("branch") else None
    x_out = v.pop("x")
    dv = doubles(v)
    args = dict(norm=norm, eps=EPS, post=post, post_eps=POST_EPS)
    ref, tol = backward_bounds(None if dy is None else f64(dy), None if do is None else f64(do), f64(x_out), group=group,
                               groups=groups, **args, **dv)
    dx = torch.full((T, D), 7.0, dtype=DTYPES[kind], device="cuda")
    dh = torch.full((T, D), 7.0, dtype=DTYPES[kind], device="cuda") if want.get("branch") else None
    ws = None
    n = L.bsq_block_norm_workspace_bytes(T, D, groups)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")   # NaN where nothing is written
    out = L.bsq_block_norm_backward(dy, do, x_out, norm=KINDS[norm], eps=EPS, post=KINDS[post], post_eps=POST_EPS,
                                    starts=st, dx=dx, dbranch=dh, workspace=ws, **v)
    live = group >= 0
    for k, t in out.items():
        if k in ("x", "branch"):
            if t is None:
                continue
            got = f64(t)
            assert np.all(np.abs(got - ref[k])[live] <= (tol[k] + rounded(ref[k], DTYPES[kind]))[live]), k
            assert np.all(got[~live] == 7.0), k
        elif v[k] is None:
            assert t is None
        else:
            assert t.dtype == torch.float32
            assert np.all(np.abs(f64(t) - ref[k]) <= tol[k] + 2.0 ** -23 * np.abs(ref[k])), k
    # asked for one by one they are the same
    for k in out:
        if out[k] is None:
            continue
        alone = L.bsq_block_norm_backward(dy, do, x_out, norm=KINDS[norm], eps=EPS, post=KINDS[post], post_eps=POST_EPS,
                                          starts=st, need=(k,), **v)
        assert torch.equal(alone[k][torch.from_numpy(live)] if k in ("x", "branch") else alone[k],
                           out[k][torch.from_numpy(live)] if k in ("x", "branch") else out[k]), k
        assert all(alone[o] is None for o in alone if o != k and not (k == "branch" and o == "x"))


def test_gradient_against_differences():
    """The kernel's gradient in fp32 along random directions, against differences of the oracle's forward in 64 bits (its
    second-order rest is below 1e-7 of the terms at this step)."""
    T, D, groups = 6, 64, 2
    v = vectors(5, T, D, "fp32", groups, **ALL)
    v["x"] *= 0.5
    dv = doubles(v)
    group, _ = groups_of(T, groups, None)
    rng = np.random.default_rng(6)
    dy, do = (torch.from_numpy(rng.standard_normal((T, D))).float().cuda() for _ in range(2))
    args = dict(eps=1e-3, post_eps=1e-3)

    def total(dv):
        o, y = block.block_norm(norm="layer", post="rms", group=group, **args, **dv)
        return (o * f64(do)).sum() + (y * f64(dy)).sum()

    x_out = torch.from_numpy(block.block_norm(norm="layer", post="rms", group=group, **args, **dv)[0]).float().cuda()
    back = {k: t for k, t in v.items() if k != "x"}
    out = L.bsq_block_norm_backward(dy, do, x_out, norm=L.BSQ_NORM_LAYER, post=L.BSQ_NORM_RMS, **args, **back)
    for k in dv:
        d = rng.standard_normal(dv[k].shape)
        up, down = dict(dv), dict(dv)
        up[k], down[k] = dv[k] + 1e-5 * d, dv[k] - 1e-5 * d
        diff = (total(up) - total(down)) / 2e-5
        got = (f64(out[k]) * d).sum()
        assert abs(diff - got) <= 2.0 ** -16 * (np.abs(f64(out[k]) * d).sum() + 1), k


def test_in_place_strides_and_broadcast():
    T, D = 33, 640
    v = vectors(1, T, D, "bf16", 1, branch=1, weight=1)
    y, _, x_out = L.bsq_block_norm(**v)
    # the stream in place, rows of a wider tensor, neighbours untouched
    wide = torch.full((T, D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + D] = v["x"]
    view = wide[:, 8:8 + D]
    y2 = torch.full((T, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    args = dict(v, x=view)
    got, _, out = L.bsq_block_norm(x_out=view, y=y2[:, D:], **args)
    assert out is view and torch.equal(view, x_out) and torch.equal(y2[:, D:], y)
    assert torch.all(y2[:, :D] == 7.0) and torch.all(wide[:, :8] == 7.0) and torch.all(wide[:, 8 + D:] == 7.0)
    # one row for all
    row = v["x"][:1].expand(T, D)
    a, _, b = L.bsq_block_norm(**dict(v, x=row))
    c, _, e = L.bsq_block_norm(**dict(v, x=row.contiguous()))
    assert torch.equal(a, c) and torch.equal(b, e)
    # gradients in place of what they come from
    dy, do = torch.randn(2, T, D, device="cuda").bfloat16()
    back = {k: t for k, t in v.items() if k != "x"}
    want = L.bsq_block_norm_backward(dy, do, x_out, post=L.BSQ_NORM_RMS, **back)
    mine, branch = do.clone(), v["branch"].clone()
    got = L.bsq_block_norm_backward(dy, mine, x_out, post=L.BSQ_NORM_RMS, dx=mine, dbranch=branch,
                                    **dict(back, branch=branch))
    assert got["x"] is mine and torch.equal(mine, want["x"]) and torch.equal(branch, want["branch"])
    mine = dy.clone()
    got = L.bsq_block_norm_backward(mine, do, x_out, post=L.BSQ_NORM_RMS, dx=mine, **back)
    assert torch.equal(mine, want["x"]) and torch.equal(got["weight"], want["weight"])


@pytest.mark.parametrize("D", [256, 2560])
def test_odd_values_stay_in_their_row(D):
    """NaN and infinities make their own row NaN and reach no other; rows of zeros are norms of zero."""
    T = 12
    v = vectors(3, T, D, "fp32", 1, branch=1, gate=1, scale=1, shift=1)
    clean = {k: None if t is None else t.clone() for k, t in v.items()}
    v["x"][2, 5], v["x"][7, 0], v["branch"][9, D - 1] = float("nan"), float("inf"), float("-inf")
    v["x"][4] = v["branch"][4] = 0.0
    rest = [0, 1, 3, 5, 6, 8, 10, 11]
    for fmt in (None, 1, 2):
        g = torch.tensor([0.01], device="cuda") if fmt == 2 else None
        a, s, _ = L.bsq_block_norm(norm=L.BSQ_NORM_LAYER, out_format=fmt, y_global=g, **v)
        b, t, _ = L.bsq_block_norm(norm=L.BSQ_NORM_LAYER, out_format=fmt, y_global=g, **clean)
        assert torch.equal(a[rest], b[rest])
        if fmt is None:
            assert torch.isnan(a[[2, 7, 9]]).all() and torch.equal(a[4], v["shift"][0])
        else:
            assert torch.equal(s[rest], t[rest])
            bad = s[[2, 7, 9]]
            assert torch.isnan(bad).all() if fmt == 1 else torch.all(bad & 0x7F == 0x7F)
    zero = torch.zeros(2, D, device="cuda")
    q, s, _ = L.bsq_block_norm(zero, out_format=L.BSQ_FMT_FP8R)
    assert torch.all(s == 0) and torch.all(q & 0x7F == 0)


def test_no_rows():
    D = 64
    e = torch.empty(0, D, device="cuda")
    y, _, x = L.bsq_block_norm(e, branch=e)
    assert y.shape == x.shape == (0, D)
    w, m = torch.ones(D, device="cuda"), torch.ones(3, D, device="cuda")
    out = L.bsq_block_norm_backward(e, e, e, weight=w, scale=m, shift=m, gate=m, branch=e, post=L.BSQ_NORM_RMS, post_weight=w)
    for k in ("weight", "post_weight", "scale", "shift", "gate"):
        assert torch.all(out[k] == 0), k
    assert out["x"].shape == (0, D)
    # rows that have no group, and groups without rows
    x, st = torch.randn(4, D, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    kept = torch.full((4, D), 7.0, device="cuda")
    L.bsq_block_norm(x, scale=m, starts=st, y=kept)
    out = L.bsq_block_norm_backward(x, None, x, weight=w, scale=m, starts=st, dx=kept)
    assert torch.all(kept == 7.0) and torch.all(out["scale"] == 0) and torch.all(out["weight"] == 0)


def test_starts_out_of_range_stay_inside():
    """What rows get for starts that decrease or leave the rows is not defined; memory around the tensors is left alone."""
    T, D, groups = 24, 1536, 4
    v = vectors(8, T, D, "bf16", groups, branch=1, gate=1, scale=1, shift=1, weight=1)
    for starts in ([5, 3, 9, 2, 400], [-9, -3, 50, 7, 24], [0, 100, 200, 300, 1 << 30], [24, 0, 24, 0, 24], [0, 8, 16, 24, -1]):
        st = torch.tensor(starts, dtype=torch.int32).cuda()
        pad = torch.full((3, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
        L.bsq_block_norm(norm=L.BSQ_NORM_LAYER, starts=st, y=pad[1], **v)
        assert torch.all(pad[0] == 7.0) and torch.all(pad[2] == 7.0)
        dy = torch.randn(T, D, device="cuda").bfloat16()
        n = L.bsq_block_norm_workspace_bytes(T, D, groups)
        ws = torch.full((n + 512,), 77, dtype=torch.uint8, device="cuda")
        back = {k: t for k, t in v.items() if k != "x"}
        L.bsq_block_norm_backward(dy, None, v["x"], norm=L.BSQ_NORM_LAYER, starts=st, dx=pad[1], workspace=ws[256:256 + n],
                                  **back)
        torch.cuda.synchronize()
        assert torch.all(pad[0] == 7.0) and torch.all(pad[2] == 7.0)
        assert torch.all(ws[:256] == 77) and torch.all(ws[256 + n:] == 77)


def test_graphs_and_streams():
    """Forward and backward captured, replayed with other rows, groups and vectors in the same buffers, between eager
    calls; and on a stream of their own."""
    T, D, groups = 100, 1280, 3
    v = vectors(4, T, D, "bf16", groups, **ALL)
    st = torch.tensor([0, 30, 60, 100], dtype=torch.int32).cuda()
    dy, do = torch.randn(2, T, D, device="cuda").bfloat16()
    args = dict(norm=L.BSQ_NORM_LAYER, post=L.BSQ_NORM_RMS, starts=st)

    def both():
        y, s, x = L.bsq_block_norm(out_format=L.BSQ_FMT_FP8R, **args, **v)
        back = {k: t for k, t in v.items() if k != "x"}
        return [y, s, x, *L.bsq_block_norm_backward(dy, do, x, **args, **back).values()]

    both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        alone = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, both()))
    graphs = []
    for _ in range(2):   # (each with its own workspace and outputs)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both()
        graphs.append((g, outs))
    for i, starts in enumerate(([0, 1, 99, 100], [0, 0, 0, 100], [0, 50, 50, 100], [0, 30, 60, 100])):
        for k, t in v.items():
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(i)))
        st.copy_(torch.tensor(starts, dtype=torch.int32))
        for g, _ in graphs:
            g.replay()
        want = both()
        torch.cuda.synchronize()
        for g, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), i


def test_offsets_past_32_bits():
    """Rows of a tensor of more than 2^32 elements, far apart."""
    T, D, stride = 5, 1024, (1 << 30) + 1024
    big = torch.zeros(4 * stride + D, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (T, D), (stride, 1))
    v = torch.randn(T, D, device="cuda").bfloat16()
    x.copy_(v)
    want = L.bsq_block_norm(v, branch=v)
    got = L.bsq_block_norm(x, branch=v, x_out=x)
    assert torch.equal(got[0], want[0]) and torch.equal(x, want[2])
    dx = L.bsq_block_norm_backward(v, None, x, need=("x",), dx=x)["x"]
    assert torch.equal(dx, L.bsq_block_norm_backward(v, None, want[2], need=("x",))["x"])


@pytest.mark.parametrize("D", [64, 1032, 4104])
def test_starts_without_vectors(D):
    """Where only starts are given, rows behind the last group are still left alone and reach no sum."""
    T = 50
    v = vectors(9, T, D, "bf16", 1, branch=1, weight=1, bias=1)
    st = torch.tensor([0, 7, 7, 41], dtype=torch.int32).cuda()
    pad = torch.full((3, T, D), 7.0, dtype=torch.bfloat16, device="cuda")
    y, _, x = L.bsq_block_norm(norm=L.BSQ_NORM_LAYER, starts=st, y=pad[0], x_out=pad[1], **v)
    part = {k: t[:41] if k in ("x", "branch") and t is not None else t for k, t in v.items()}
    want = L.bsq_block_norm(norm=L.BSQ_NORM_LAYER, **part)
    assert torch.equal(y[:41], want[0]) and torch.equal(x[:41], want[2]) and torch.all(pad[:2, 41:] == 7.0)
    dy = torch.randn(T, D, device="cuda").bfloat16()
    dy[41:] = float("nan")
    back = {k: t for k, t in v.items() if k != "x"}
    got = L.bsq_block_norm_backward(dy, None, x, norm=L.BSQ_NORM_LAYER, starts=st, dx=pad[2], **back)
    group = np.where(np.arange(T) < 41, 0, -1)
    clean = np.nan_to_num(f64(dy))
    ref, tol = backward_bounds(clean, None, f64(x), "layer", EPS, group, 1, **doubles(back))
    for k in ("weight", "bias"):
        assert np.all(np.abs(f64(got[k]) - ref[k]) <= tol[k] + 2.0 ** -23 * np.abs(ref[k])), k
    assert torch.all(pad[2, 41:] == 7.0)
    assert np.all(np.abs(f64(got["x"]) - ref["x"])[:41] <= (tol["x"] + rounded(ref["x"], torch.bfloat16))[:41])


@pytest.mark.parametrize("T,groups", [(64, 64), (130, 65), (900, 3), (66000, 66000)])
def test_sums_of_all_groups(T, groups):
    """The gradients that all groups share, along with the groups' own and after them, and asked for alone."""
    D = 64
    v = vectors(T, T, D, "fp32", groups, **ALL)
    group = np.arange(T) // (T // groups)
    dy, do = torch.randn(2, T, D, generator=torch.Generator().manual_seed(T)).cuda()
    x_out = v.pop("x")
    dv = doubles(v)
    args = dict(norm="layer", eps=EPS, post="rms", post_eps=POST_EPS)
    if groups > 1000:   # (the oracle's sums by groups are a product with all of them: take those of the shared alone)
        D_all = {k: t for k, t in dv.items()}
        spread = {k: D_all[k][group] for k in ("scale", "shift", "gate")}
        n = block.normed(f64(x_out), "layer", EPS)[0]
        d = f64(dy) * (1 + spread["scale"])
        got = L.bsq_block_norm_backward(dy, do, x_out, norm=L.BSQ_NORM_LAYER, eps=EPS, post=L.BSQ_NORM_RMS, post_eps=POST_EPS, **v)
        chain = (T / 512 + groups / 128 + 64) * 2.0 ** -24 + 2.0 ** -16   # (2^-16: the errors of N, a term's at most)
        assert np.all(np.abs(f64(got["weight"]) - (d * n).sum(0)) <= chain * np.abs(d * n).sum(0) + 2.0 ** -14 * np.abs(d).sum(0))
        assert np.all(np.abs(f64(got["bias"]) - d.sum(0)) <= chain * np.abs(d).sum(0))
        assert np.all(np.abs(f64(got["shift"]) - f64(dy)) == 0.0)
        return
    ref, tol = backward_bounds(f64(dy), f64(do), f64(x_out), group=group, groups=groups, **args, **dv)
    call = lambda **kw: L.bsq_block_norm_backward(dy, do, x_out, norm=L.BSQ_NORM_LAYER, eps=EPS, post=L.BSQ_NORM_RMS,  # noqa: E731
                                                  post_eps=POST_EPS, **v, **kw)
    out = call()
    for k in ("scale", "shift", "gate", "weight", "bias", "post_weight"):
        assert np.all(np.abs(f64(out[k]) - ref[k]) <= tol[k] + 2.0 ** -23 * np.abs(ref[k])), k
    alone = call(need=("weight", "bias", "post_weight"))
    assert all(torch.equal(alone[k], out[k]) for k in ("weight", "bias", "post_weight")) and alone["x"] is None


@pytest.mark.parametrize("T,groups", [(40, 5), (300, 70)])
def test_vectors_of_groups_without_rows_do_not_count(T, groups):
    """They may hold anything: the same gradients as with ones there, and zeros for the groups themselves, whatever the
    vectors that all share hold."""
    D = 776
    v = vectors(11, T, D, "fp32", groups, branch=1, gate=1, scale=1, shift=1, weight=1, bias=1, post_weight=1)
    n = [T // 2 if g in (1, 3) else 0 for g in range(groups)]
    st = torch.tensor([0, *np.cumsum(n)], dtype=torch.int32).cuda()
    without = torch.tensor([k == 0 for k in n], device="cuda")
    dy, x = torch.randn(T, D, device="cuda"), v.pop("x")
    outs = []
    for fill in (1.0, float("nan")):
        for k in ("gate", "scale", "shift"):
            v[k][without] = fill
        outs.append(L.bsq_block_norm_backward(dy, x, x, norm=L.BSQ_NORM_LAYER, post=L.BSQ_NORM_RMS, starts=st, **v))
    for k, t in outs[0].items():
        assert torch.isfinite(t).all() and torch.equal(t, outs[1][k]), k
    for k in ("weight", "bias", "post_weight"):
        v[k][5] = float("inf")
    out = L.bsq_block_norm_backward(dy, x, x, norm=L.BSQ_NORM_LAYER, post=L.BSQ_NORM_RMS, starts=st, **v)
    for k in ("gate", "scale", "shift"):
        assert torch.all(out[k][without] == 0), k
