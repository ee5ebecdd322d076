"""GPU tests of the block norms' forms that test_gpu_block_norm.py does not run: the gated residual alone, one group among
many that holds almost all rows, inputs that are one row for all, calls on two streams at once. Tolerances as derived in
tests/block_util.py; for the sums of a long group see below."""
import numpy as np
import pytest
import torch

from oracle import block
from tests.block_util import DTYPES, backward_bounds, f64, forward_bounds, rounded
from tests.test_gpu_block_norm import ALL, EPS, KINDS, POST_EPS, doubles, groups_of, vectors

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,D,post,groups,starts,want", [
    (1, 8, None, 1, None, {}),
    (5, 72, "rms", 3, [0, 0, 3, 5], dict(gate=1, post_weight=1)),
    (67, 512, "layer", 1, None, {}),
    (66, 520, None, 2, None, dict(gate=1)),
    (130, 1536, None, 3, [0, 7, 7, 121], dict(gate=1)),
    (24, 2560, "layer", 24, None, dict(gate=1, post_weight=1)),
    (7, 5120, "rms", 2, [0, 3, 5], dict(gate=1)),
    (3, 8192, None, 1, [0, 2], {}),
    (4, 16384, "layer", 2, None, dict(gate=1, post_weight=1)),
    (9000, 64, "rms", 3, [0, 1, 8000, 8999], dict(gate=1, post_weight=1))])
def test_gated_residual_alone(T, D, post, groups, starts, want, kind):
    v = {k: t for k, t in vectors(T + D, T, D, kind, groups, branch=1, **want).items()
         if k in ("x", "branch", "gate", "post_weight")}
    group, st = groups_of(T, groups, starts)
    out, eo, _, _ = forward_bounds(norm=None, eps=EPS, post=post, post_eps=POST_EPS, group=group, **doubles(v))
    live = group >= 0
    args = dict(norm=L.BSQ_NORM_NONE, eps=EPS, post=KINDS[post], post_eps=POST_EPS, starts=st)
    buf = torch.full((T, D), 7.0, dtype=DTYPES[kind], device="cuda")
    y, s, got = L.bsq_block_norm(x_out=buf, **args, **v)
    assert y is None and s is None and got is buf
    assert np.all(np.abs(f64(got) - out)[live] <= (eo + rounded(out, DTYPES[kind]))[live])
    assert np.all(f64(got)[~live] == 7.0)
    # the same as beside a norm, and in place, rows of a wider tensor
    assert torch.equal(L.bsq_block_norm(x_out=buf.clone(), **dict(args, norm=L.BSQ_NORM_RMS), **v)[2], got)
    wide = torch.full((T, D + 16), 3.0, dtype=DTYPES[kind], device="cuda")
    wide[:, 8:8 + D] = v["x"]
    L.bsq_block_norm(x_out=wide[:, 8:8 + D], **args, **dict(v, x=wide[:, 8:8 + D]))
    assert torch.equal(wide[:, 8:8 + D][live], got[live]) and torch.equal(wide[:, 8:8 + D][~live], v["x"][~live])
    assert torch.all(wide[:, :8] == 3.0) and torch.all(wide[:, 8 + D:] == 3.0)
    # one branch for all rows
    one = dict(v, branch=v["branch"][:1].expand(T, D))
    a = L.bsq_block_norm(x_out=buf.clone(), **args, **one)[2]
    b = L.bsq_block_norm(x_out=buf.clone(), **args, **dict(one, branch=one["branch"].contiguous()))[2]
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,D,groups", [(20_000, 512, 200), (6000, 1536, 130), (3000, 4096, 40)])
def test_one_group_holds_almost_all_rows(T, D, groups):
    """Its slots are added by as few threads of a column as those of groups with one row. A sum passes the rows of a worker
    (4 here, or T / (256 x 12) rounded up, 7 for the first), the slots of the group (one a worker) in 8 threads, 3 steps over
    lanes, and for what all groups share the groups in at most 128 threads with 3 + 16 steps more: at most
    7 + 20000 / 7 / 8 + 30 = 395, 4 + 1500 / 8 + 35 = 227 and 4 + 750 / 8 + 35 + 40 = 173 additions of 2^-24 each."""
    chain = {20_000: 395, 6000: 227, 3000: 173}[T] * 2.0 ** -24
    v = vectors(T, T, D, "fp32", groups, **ALL)
    big = groups // 2
    sizes = [0 if g % 7 == 3 else 1 for g in range(groups)]
    sizes[big] = T - 5 - sum(sizes) + sizes[big]
    starts = [0, *np.cumsum(sizes).tolist()]
    group, st = groups_of(T, groups, starts)
    dy, do = torch.randn(2, T, D, generator=torch.Generator().manual_seed(T)).cuda()
    x_out = v.pop("x")
    dv = doubles(v)
    args = dict(norm="layer", eps=EPS, post="rms", post_eps=POST_EPS)
    ref, tol = backward_bounds(f64(dy), f64(do), f64(x_out), group=group, groups=groups, **args, **dv)
    out = L.bsq_block_norm_backward(dy, do, x_out, norm=L.BSQ_NORM_LAYER, eps=EPS, post=L.BSQ_NORM_RMS, post_eps=POST_EPS,
                                    starts=st, **v)
    live = group >= 0
    member = np.zeros((groups, T))
    member[group[live], np.nonzero(live)[0]] = 1.0
    n, h = block.normed(f64(x_out), "layer", EPS)[0], block.normed(dv["branch"], "rms", POST_EPS)[0]
    d, c = np.abs(f64(dy)), np.abs(ref["x"])
    s, g = np.abs(1 + block._rows(dv["scale"], group, 0.0, D)), np.abs(block._rows(dv["gate"], group, 1.0, D))
    terms = {"scale": member @ (d * (np.abs(n * dv["weight"]) + np.abs(dv["bias"]))), "shift": member @ d,
             "gate": member @ (c * np.abs(h * dv["post_weight"])), "weight": (s * d * np.abs(n))[live].sum(0),
             "bias": (s * d)[live].sum(0), "post_weight": (g * c * np.abs(h))[live].sum(0)}
    for k, t in terms.items():
        assert np.all(np.abs(f64(out[k]) - ref[k]) <= tol[k] + chain * t + 2.0 ** -23 * np.abs(ref[k])), k
    again = L.bsq_block_norm_backward(dy, do, x_out, norm=L.BSQ_NORM_LAYER, eps=EPS, post=L.BSQ_NORM_RMS, post_eps=POST_EPS,
                                      starts=st, **v)
    assert all(torch.equal(out[k][torch.from_numpy(live)] if k in ("x", "branch") else out[k],
                           again[k][torch.from_numpy(live)] if k in ("x", "branch") else again[k]) for k in out)


@pytest.mark.parametrize("D", [64, 1032, 8192])
def test_one_row_for_all_in_the_gradient(D):
    T = 41
    v = vectors(2, T, D, "bf16", 1, branch=1, weight=1, gate=1, post_weight=1)
    dy, do = torch.randn(2, T, D, device="cuda").bfloat16()
    x_out, b = v.pop("x"), v.pop("branch")
    row = lambda t: t[:1].expand(T, D)  # noqa: E731
    call = lambda f: L.bsq_block_norm_backward(f(dy), f(do), f(x_out), norm=L.BSQ_NORM_LAYER, post=L.BSQ_NORM_RMS,  # noqa: E731
                                               branch=f(b), **v)
    a, c = call(row), call(lambda t: row(t).contiguous())
    for k in a:
        assert (a[k] is None and c[k] is None) or torch.equal(a[k], c[k]), k


def test_two_streams_at_once():
    """Norms, their gradients and linears on two streams, each with its own tensors: the bits of one after the other."""
    T, D = 700, 1024
    sets = []
    for seed in (1, 2):
        v = vectors(seed, T, D, "bf16", 3, **ALL)
        st = torch.tensor([0, 100 * seed, 500, T], dtype=torch.int32).cuda()
        dy, do = torch.randn(2, T, D, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        w, ws = L.bsq_quantize_act_fp8r(torch.randn(D, D, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda())
        sets.append((v, st, dy, do, w, ws))

    def run(v, st, dy, do, w, ws):
        q, s, x = L.bsq_block_norm(norm=L.BSQ_NORM_LAYER, post=L.BSQ_NORM_RMS, starts=st, out_format=L.BSQ_FMT_FP8R, **v)
        back = {k: t for k, t in v.items() if k != "x"}
        g = L.bsq_block_norm_backward(dy, do, x, norm=L.BSQ_NORM_LAYER, post=L.BSQ_NORM_RMS, starts=st, **back)
        y = L.bsq_gemm_fp8r_q_epilogue(q, s, w, ws, act=L.BSQ_ACT_GELU, gate=v["gate"], residual=x, starts=st)
        return [q, s, x, *g.values(), y]

    want = [run(*a) for a in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))
