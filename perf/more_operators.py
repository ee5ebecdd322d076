"""Cases, plain forms and exact values of the operators of a transformer block around its quantized linears: rotary
positions with several axes, the gated residual with the norm before and after it (and its gradient), and linears with
bias, activation, gate and residual in their epilogue.

own = False: run() computes the operators with elementary torch operations in 32 bits;
own = True:  run() makes the calls of block_scaled_precision_row_amd._lib.

Rows are packed: with ragged groups, group g has rows starts[g] .. starts[g + 1] - 1 and its own vectors of scale, shift
and gate; otherwise the rows are split evenly.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0
EPS = 1e-6


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # queries and keys of one small image tile, rows and columns as two axes: latency
        _rope("rope_tile", 64, 32, 128, [32, 32], "blocks", "half", "bf16", False),
        # queries and keys of a clip (time, rows, columns), neighbouring elements as pairs
        _rope("rope_clip", 14_400, 48, 128, [8, 28, 28], "blocks", "interleaved", "bf16", False),
        # the gradient of the rotation with the axes taken in turn, half of each head turned, in fp32
        _rope("rope_grad", 5001, 24, 128, [12, 10, 10], "cycled", "half", "fp32", True),
        # a few tokens of a decoder: the branch normed, added, and the next block's norm
        _norm("norm_step", 24, 4096, "rms", "fp16", weight=True, branch=True, post=True),
        # an image's tokens between two blocks: gated residual, norm, scale and shift, rows encoded for an fp8r linear
        _norm("norm_image", 8192, 5120, "layer", "bf16", branch=True, gate=True, mod=True, groups=2, out="fp8r"),
        # its gradient in training, images of several sizes packed
        _norm("norm_grad", 4608, 2560, "layer", "bf16", branch=True, gate=True, mod=True, groups=5, ragged=True,
              backward=True),
        # the gradient of a norm with weights after and before a branch, in fp32
        _norm("norm_grad_weights", 1001, 1536, "rms", "fp32", weight=True, branch=True, post=True, backward=True),
        # the embedding of a time step of two images: bias and activation, latency
        _linear("linear_step", "fp8r", 2, 5120, 2560, act="silu"),
        # a decode batch through a projection that is added to the residual
        _linear("linear_few", "nvfp4", 24, 4096, 4096, residual=True),
        # an image's tokens up to the inner width, with the activation
        _linear("linear_up", "fp8r", 4096, 10_240, 2560, act="gelu_tanh"),
        # and back down into the gated residual, images of several sizes packed
        _linear("linear_down", "nvfp4", 4608, 2560, 10_240, residual=True, gate=True, groups=5, ragged=True),
        # an odd crop with odd widths
        _linear("linear_odd", "fp8r", 777, 1234, 1056, act="gelu", residual=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "norm", "norm", "linear", "linear"])
    if op == "rope":
        dim = rng.choice([64, 128, 128, 256])
        pairs, axes = rng.choice([dim // 2, dim // 2, dim // 4]), rng.choice([2, 3, 3])
        rest = [pairs // (2 * axes) + rng.randint(0, pairs // (2 * axes)) for _ in range(axes - 1)]
        kind = rng.choice(["bf16", "fp16", "fp32"])
        return _rope(None, spread(1, 14_400), rng.randint(1, (6144 if kind != "fp32" else 3070) // dim), dim,
                     [pairs - sum(rest)] + rest, rng.choice(["blocks", "cycled"]), rng.choice(["half", "interleaved"]),
                     kind, rng.random() < 0.4)
    if op == "norm":
        backward, branch, mod = rng.random() < 0.5, rng.random() < 0.8, rng.random() < 0.6
        kind, groups = rng.choice(["bf16", "fp16", "fp32"]), rng.randint(1, 6) if mod else 1
        out = rng.choice([None, "fp8r"]) if not backward else None
        dim = 32 * spread(4, 160)
        most = (140_000_000 // 6 if backward else 290_000_000 // 4) // (4 if kind == "fp32" else 2) // dim
        return _norm(None, spread(groups, min(most, 16_384)), dim, rng.choice(["rms", "layer"]), kind,
                     weight=rng.random() < 0.5, branch=branch, post=branch and rng.random() < 0.4,
                     gate=branch and mod and rng.random() < 0.7, mod=mod, groups=groups, ragged=mod and rng.random() < 0.7,
                     backward=backward, out=out)
    fmt, residual = rng.choice(["fp8r", "nvfp4"]), rng.random() < 0.6
    gate, tokens = residual and rng.random() < 0.5, rng.choice([spread(1, 128), spread(64, 4608)])
    most = min(10_240, (28_000_000 if residual else 41_000_000) // tokens)
    n = rng.choice([spread(64, most), 64 * spread(1, most // 64)])
    k = 32 * spread(2, max(3, min(320, 4608 * 2560 * 10_240 // (tokens * n) // 32)))
    return _linear(None, fmt, tokens, n, k, act=rng.choice(["none", "gelu_tanh", "gelu", "silu"]),
                   residual=residual, gate=gate, groups=rng.randint(1, min(6, tokens)) if gate else 1, ragged=gate)


def _named(name, case):
    return dict(case, name=name) if name else case


def _rope(name, tokens, heads, dim, sections, order, layout, kind, backward):
    """sections: the pairs of each axis, as a text ("8,28,28")."""
    return _named(name, {"op": "rope", "tokens": tokens, "heads": heads, "dim": dim,
                         "sections": ",".join(map(str, sections)), "order": order, "layout": layout, "type": kind,
                         "backward": backward})


def _norm(name, rows, dim, norm, kind, weight=False, branch=False, post=False, gate=False, mod=False, groups=1,
          ragged=False, backward=False, out=None):
    return _named(name, {"op": "norm_grad" if backward else "norm", "rows": rows, "dim": dim, "norm": norm, "type": kind,
                         "weight": weight, "branch": branch, "post": post, "gate": gate, "mod": mod, "groups": groups,
                         "ragged": ragged, "out": out or "plain"})


def _linear(name, fmt, rows, n, k, act="none", residual=False, gate=False, groups=1, ragged=False):
    return _named(name, {"op": "linear", "format": fmt, "rows": rows, "n": n, "k": k, "act": act, "residual": residual,
                         "gate": gate, "groups": groups, "ragged": ragged})


# ---- inputs --------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"rope": _prepare_rope, "norm": _prepare_norm, "norm_grad": _prepare_norm,
            "linear": _prepare_linear}[case["op"]](case, g, {"case": case})


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _axis_of_pair(case):
    """blocks: the first sections[0] pairs turn with axis 0 and so on; cycled: pair i with axis i % axes while that axis
    has pairs left (i / axes < its section), and with axis 0 otherwise."""
    sections = _sections(case)
    if case["order"] == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    axes = len(sections)
    return [i % axes if i // axes < sections[i % axes] else 0 for i in range(sum(sections))]


def _prepare_rope(case, g, state):
    sections, T = _sections(case), case["tokens"]
    x = torch.randn(T, case["heads"], case["dim"], generator=g, device="cuda").to(TYPES[case["type"]])
    # a grid of this many tokens, walked along the last axis first, somewhere in a larger one
    side = max(1, math.ceil(T ** (1 / len(sections))))
    t = torch.arange(T, device="cuda")
    places = [t // side ** k % side for k in reversed(range(len(sections)))]
    positions = torch.stack(places, -1) + torch.randint(0, 2000, (len(sections),), generator=g, device="cuda")
    if case["order"] == "blocks":  # each axis has frequencies of its own
        f = torch.cat([10_000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections])
    else:                          # one run of frequencies, shared out among the axes
        f = 1_000_000.0 ** (-torch.arange(sum(sections), dtype=torch.float64) / sum(sections))
    state.update(x=x, positions=positions, inv_freq=f.float().cuda(), y=torch.empty_like(x), sections=sections,
                 axis=torch.tensor(_axis_of_pair(case)).cuda())
    return state


def _starts(case):
    """Where each group of rows starts: the case's own, so that outputs of all inputs have one shape."""
    rows, groups = case["rows"], case["groups"]
    g = torch.Generator()
    g.manual_seed(1000 * groups + rows)
    cuts = torch.randperm(rows - 1, generator=g)[:groups - 1].sort().values + 1 if groups > 1 else torch.zeros(0)
    return [0] + [int(c) for c in cuts] + [rows]


def _groups(case, state):
    """ragged: the groups' starts; otherwise a number of groups that divides the rows."""
    if case["ragged"]:
        state["starts"] = torch.tensor(_starts(case), dtype=torch.int32).cuda()
        return case["groups"]
    state["starts"] = None
    return math.gcd(case["rows"], case["groups"])


def _prepare_norm(case, g, state):
    T, D, kind = case["rows"], case["dim"], TYPES[case["type"]]

    def normal(*shape, size=1.0, mean=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * size + mean).to(kind)

    n = _groups(case, state)
    # a residual stream: some channels much larger than the others, a mean that is not zero
    loud = 1 + 20 * (torch.rand(D, generator=g, device="cuda") < 0.01)
    state["x"] = (torch.randn(T, D, generator=g, device="cuda") * 2 * loud + 0.3).to(kind)
    mod = normal(n, 3 * D, size=0.5) if case["mod"] or case["gate"] else None  # as a modulation linear writes them
    state.update(
        branch=normal(T, D, size=0.7) if case["branch"] else None,
        scale=mod[:, :D] if case["mod"] else None, shift=mod[:, D:2 * D] if case["mod"] else None,
        gate=mod[:, 2 * D:] if case["gate"] else None,
        weight=normal(D, size=0.3, mean=1.0) if case["weight"] else None,
        bias=normal(D, size=0.3) if case["weight"] and case["norm"] == "layer" else None,
        post_weight=normal(D, size=0.3, mean=0.5) if case["post"] else None)
    if case["op"] == "norm":
        state["x_out"] = torch.empty_like(state["x"]) if case["branch"] else None
        if case["out"] == "fp8r":
            state.update(y=torch.empty(T, D, dtype=torch.uint8, device="cuda"), y_scale=torch.empty(T, device="cuda"))
        else:
            state["y"] = torch.empty_like(state["x"])
    else:
        state.update(dy=normal(T, D, size=0.01), dx_out=normal(T, D, size=0.01) if case["branch"] else None)
    return state


def _codes(shape, g, size):
    return (torch.randn(shape, generator=g, device="cuda") * size).clamp(-E4M3_MAX, E4M3_MAX).to(
        torch.float8_e4m3fn).view(torch.uint8)


def _prepare_linear(case, g, state):
    M, N, K = case["rows"], case["n"], case["k"]
    n = _groups(case, state)
    # activations and weights as the quantizers leave them, so that outputs are of order one
    if case["format"] == "fp8r":
        state.update(xq=_codes((M, K), g, 110.0), w=_codes((N, K), g, 110.0),
                     x_scale=torch.rand(M, generator=g, device="cuda") * 0.01 + 0.005,
                     w_scale=(torch.rand(N, generator=g, device="cuda") + 0.5) / (110.0 * math.sqrt(K)))
    else:
        def blocks(rows):
            return (torch.rand(rows, K // 16, generator=g, device="cuda") * 200 + 100).to(torch.float8_e4m3fn).view(
                torch.uint8)
        state.update(xq=torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                     w=torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                     x_scale=blocks(M), w_scale=blocks(N), input_scale=torch.full((1,), 1 / 600.0, device="cuda"),
                     w_scale2=torch.full((1,), 1 / (600.0 * math.sqrt(K)), device="cuda"))

    def normal(*shape, size=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * size).to(torch.bfloat16)

    state.update(bias=normal(N, size=0.5), residual=normal(M, N, size=2.0) if case["residual"] else None,
                 gate=normal(n, N, size=0.5) if case["gate"] else None,
                 y=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    return state


# ---- one pass ------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"rope": _plain_rope, "norm": _plain_norm, "norm_grad": _plain_norm_grad,
            "linear": _plain_linear}[case["op"]](case, state)


def _own(case, s):
    from block_scaled_precision_row_amd import _lib as L
    if case["op"] == "rope":
        return L.bsq_rope_axes(s["x"], s["positions"], s["inv_freq"], s["sections"],
                               L.BSQ_AXES_CYCLED if case["order"] == "cycled" else L.BSQ_AXES_BLOCKS,
                               L.BSQ_ROPE_INTERLEAVED if case["layout"] == "interleaved" else L.BSQ_ROPE_HALF,
                               backward=case["backward"], y=s["y"])
    if case["op"] == "linear":
        act = {"none": L.BSQ_ACT_NONE, "gelu_tanh": L.BSQ_ACT_GELU_TANH, "gelu": L.BSQ_ACT_GELU,
               "silu": L.BSQ_ACT_SILU}[case["act"]]
        more = {"bias": s["bias"], "act": act, "gate": s["gate"], "residual": s["residual"], "starts": s["starts"],
                "y": s["y"]}
        if case["format"] == "fp8r":
            return L.bsq_gemm_fp8r_q_epilogue(s["xq"], s["x_scale"], s["w"], s["w_scale"], **more)
        return L.bsq_gemm_nvfp4_q_epilogue(s["xq"], s["x_scale"], s["input_scale"], s["w"], s["w_scale"], s["w_scale2"],
                                           **more)
    kind = L.BSQ_NORM_RMS if case["norm"] == "rms" else L.BSQ_NORM_LAYER
    post = L.BSQ_NORM_RMS if case["post"] else L.BSQ_NORM_NONE
    if case["op"] == "norm":
        y, y_scale, x = L.bsq_block_norm(
            s["x"], kind, EPS, s["weight"], s["bias"], s["scale"], s["shift"], s["branch"], s["gate"], post,
            s["post_weight"], s["starts"], out_format=L.BSQ_FMT_FP8R if case["out"] == "fp8r" else None, y=s["y"],
            y_scale=s.get("y_scale"), x_out=s["x_out"])
        if case["out"] == "fp8r":
            y = y.view(torch.float8_e4m3fn)
        return {"y": y, "y_scale": y_scale, "x": x if case["branch"] else None}
    return L.bsq_block_norm_backward(s["dy"], s["dx_out"], s["x"], kind, EPS, s["weight"], s["bias"], s["scale"],
                                     s["shift"], s["branch"], s["gate"], post, s["post_weight"], s["starts"])


def _plain_rope(case, s):
    pairs = s["inv_freq"].numel()
    angle = s["positions"][:, s["axis"]].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if case["backward"]:
        sin = -sin
    x = s["x"].float()
    r = x[..., :2 * pairs]
    if case["layout"] == "half":
        a, b = r[..., :pairs], r[..., pairs:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    s["y"].copy_(torch.cat([r, x[..., 2 * pairs:]], -1))
    return s["y"]


def _group_of_row(s, rows, groups):
    if s["starts"] is None:
        return torch.arange(rows, device="cuda") // (rows // groups)
    return torch.searchsorted(s["starts"], torch.arange(rows, device="cuda", dtype=torch.int32), right=True) - 1


def _per_row(v, group):
    return None if v is None else v.float()[group]


def _normed(x, kind):
    """x normed along its rows, and the reciprocal of its size."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _vectors(case, s):
    """The groups' vectors laid out for each row, and the group of each row."""
    some = s["scale"] if s["scale"] is not None else s["gate"]
    group = None if some is None else _group_of_row(s, case["rows"], some.shape[0])
    return _per_row(s["scale"], group), _per_row(s["shift"], group), _per_row(s["gate"], group), group


def _plain_norm(case, s):
    scale, shift, gate, _ = _vectors(case, s)
    x = s["x"].float()
    if case["branch"]:
        h = s["branch"].float()
        if case["post"]:
            h = _normed(h, "rms")[0] * s["post_weight"].float()
        x = x + (h if gate is None else gate * h)
        s["x_out"].copy_(x)
    y = _normed(x, case["norm"])[0]
    if s["weight"] is not None:
        y = y * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if case["mod"]:
        y = y * (1 + scale) + shift
    if case["out"] == "fp8r":
        s["y_scale"].copy_(y.abs().amax(-1) / E4M3_MAX)
        r = torch.where(s["y_scale"] > 0, 1 / s["y_scale"], 0.0)
        y = (y * r[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["y"].copy_(y.view(torch.uint8))
        return {"y": s["y"].view(torch.float8_e4m3fn), "y_scale": s["y_scale"], "x": s["x_out"]}
    s["y"].copy_(y)
    return {"y": s["y"], "y_scale": None, "x": s["x_out"] if case["branch"] else None}


def _through_norm(d, n, r, kind):
    """The gradient of x for d, that of its normed values n = (x - mean) r."""
    d = d - n * (d * n).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - d.mean(-1, keepdim=True)
    return d * r


def _plain_norm_grad(case, s):
    """Of x_out = x + gate post(branch), y = (norm(x_out) weight + bias) (1 + scale) + shift, for the gradients of y and
    of x_out; s["x"] is x_out."""
    kind = TYPES[case["type"]]
    scale, _, gate, group = _vectors(case, s)
    dy, (n, r) = s["dy"].float(), _normed(s["x"].float(), case["norm"])
    out = dict.fromkeys(("x", "branch", "gate", "scale", "shift", "weight", "bias", "post_weight"))
    weight = None if s["weight"] is None else s["weight"].float()
    if group is not None:
        groups = (s["scale"] if s["scale"] is not None else s["gate"]).shape[0]
        member = (group == torch.arange(groups, device="cuda")[:, None]).float()
    if case["mod"]:
        m = n if weight is None else n * weight
        if s["bias"] is not None:
            m = m + s["bias"].float()
        out["scale"], out["shift"] = member @ (dy * m), member @ dy
        dy = dy * (1 + scale)
    if weight is not None:
        out["weight"] = (dy * n).sum(0)
        if s["bias"] is not None:
            out["bias"] = dy.sum(0)
        dy = dy * weight
    dx = _through_norm(dy, n, r, case["norm"])
    if case["branch"]:
        dx = dx + s["dx_out"].float()
        h = s["branch"].float()
        if case["post"]:
            hn, hr = _normed(h, "rms")
            h = hn * s["post_weight"].float()
        dh = dx
        if gate is not None:
            out["gate"] = member @ (dx * h)
            dh = dx * gate
        if case["post"]:
            out["post_weight"] = (dh * hn).sum(0)
            dh = _through_norm(dh * s["post_weight"].float(), hn, hr, "rms")
        out["branch"] = dh.to(kind)
    out["x"] = dx.to(kind)
    return out


def _e2m1(packed):
    """Packed E2M1 codes, the even element in the low nibble, as fp32 values."""
    c = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    e, m = ((c >> 1) & 3).float(), (c & 1).float()
    v = torch.where(e > 0, torch.exp2(e - 1) * (1 + 0.5 * m), 0.5 * m)
    return torch.where(c > 7, -v, v)


def _plain_linear(case, s):
    if case["format"] == "fp8r":
        x, w = s["xq"].view(torch.float8_e4m3fn).float(), s["w"].view(torch.float8_e4m3fn).float()
        y = x @ w.t() * s["x_scale"][:, None] * s["w_scale"]
    else:
        x, w = ((_e2m1(c).view(c.shape[0], -1, 16) * b.view(torch.float8_e4m3fn).float()[..., None]).flatten(1)
                for c, b in ((s["xq"], s["x_scale"]), (s["w"], s["w_scale"])))
        y = x @ w.t() * (s["input_scale"] * s["w_scale2"])
    y = y + s["bias"].float()
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    if case["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if case["act"] == "gelu":
        y = 0.5 * y * torch.special.erfc(-y * math.sqrt(0.5))
    if s["gate"] is not None:
        y = y * s["gate"].float()[_group_of_row(s, case["rows"], s["gate"].shape[0])]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["y"].copy_(y)
    return s["y"]


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
        sections = _sections(case)
        return {"bytes": 2 * n * size + 8 * len(sections) * case["tokens"], "flops": 3 * n * 2 * sum(sections) // case["dim"]}
    groups = case["groups"] if case["ragged"] else math.gcd(case["rows"], case["groups"])
    if case["op"] == "linear":
        M, N, K = case["rows"], case["n"], case["k"]
        codes = (M + N) * K if case["format"] == "fp8r" else (M + N) * (K // 2 + K // 16)
        more = (2 * M * N if case["residual"] else 0) + (2 * groups * N if case["gate"] else 0)
        return {"bytes": codes + 2 * M * N + 2 * N + more, "flops": 2 * M * N * K}
    size, n = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]], case["rows"] * case["dim"]
    vectors = groups * case["dim"] * ((2 if case["mod"] else 0) + (1 if case["gate"] else 0))
    if case["op"] == "norm":
        out = 1 if case["out"] == "fp8r" else size
        return {"bytes": n * (size + out + (2 * size if case["branch"] else 0)) + vectors * size, "flops": 12 * n}
    # reads dy and x, and with a branch dx_out and the branch (which its own gradient needs only for a gate or a norm)
    reads = 2 + (1 + (case["gate"] or case["post"]) if case["branch"] else 0)
    writes = 2 if case["gate"] or case["post"] else 1
    return {"bytes": n * size * (reads + writes) + vectors * (size + 4), "flops": 20 * n}


# ---- exact values, from the definitions, in 64 bits ----------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "linear":
        return _exact_linear(case, s)
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_norm_grad(case, s)


def _exact_rope(case, s):
    pairs, sections = s["inv_freq"].numel(), _sections(case)
    where = torch.zeros(case["tokens"], pairs, dtype=torch.float64, device="cuda")
    at = 0
    for a, n in enumerate(sections):
        p = s["positions"][:, a].double()[:, None]
        if case["order"] == "blocks":
            where[:, at:at + n] = p
            at += n
        elif a == 0:
            where[:] = p
        else:
            where[:, a:len(sections) * n:len(sections)] = p
    turn = torch.polar(torch.ones_like(where), (-1.0 if case["backward"] else 1.0) * where * s["inv_freq"].double())
    y = s["x"].double().clone()
    if case["layout"] == "half":
        z = torch.complex(y[..., :pairs], y[..., pairs:2 * pairs]) * turn[:, None]
        y[..., :pairs], y[..., pairs:2 * pairs] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]) * turn[:, None]
        y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2] = z.real, z.imag
    return y


def _slices(case):
    if case["ragged"]:
        starts = _starts(case)
        return [slice(a, b) for a, b in zip(starts[:-1], starts[1:])]
    n = case["rows"] // math.gcd(case["rows"], case["groups"])
    return [slice(a, a + n) for a in range(0, case["rows"], n)]


def _definition(case, v):
    """(x_out, y) group by group, from the inputs in `v` in 64 bits."""
    streams, outs = [], []
    for g, rows in enumerate(_slices(case)):
        x = v["x"][rows]
        if case["branch"]:
            h = v["branch"][rows]
            if case["post"]:
                h = h / torch.sqrt(h.square().sum(-1, keepdim=True) / case["dim"] + EPS) * v["post_weight"]
            x = x + (v["gate"][g] * h if case["gate"] else h)
        streams.append(x)
        if case["norm"] == "layer":
            n = (x - x.mean(-1, keepdim=True)) / torch.sqrt(x.var(-1, keepdim=True, unbiased=False) + EPS)
        else:
            n = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["dim"] + EPS)
        n = n * v["weight"] if v["weight"] is not None else n
        n = n + v["bias"] if v["bias"] is not None else n
        outs.append(n * (v["scale"][g] + 1) + v["shift"][g] if case["mod"] else n)
    return torch.cat(streams), torch.cat(outs)


_INPUTS = ("x", "branch", "gate", "scale", "shift", "weight", "bias", "post_weight")


def _doubles(s):
    return {k: None if s[k] is None else s[k].double() for k in _INPUTS}


def _nearest_e4m3(x):
    """The E4M3 value nearest to x (ties to even), in fp64: steps of an eighth of x's power of two, at least 2^-9."""
    power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(power - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(case, s):
    x, y = _definition(case, _doubles(s))
    scale = None
    if case["out"] == "fp8r":
        scale = y.abs().amax(-1) / E4M3_MAX
        y = _nearest_e4m3(y / scale[:, None])
    return {"y": y, "y_scale": scale, "x": x if case["branch"] else None}


def _exact_norm_grad(case, s):
    """By differentiation of the definition in 64 bits. s["x"] is x_out, so x is what the branch leaves of it."""
    v = _doubles(s)
    if case["branch"]:
        v["x"] = v["x"] - _definition(case, dict(v, x=torch.zeros_like(v["x"])))[0]
    for k in _INPUTS:
        if v[k] is not None:
            v[k].requires_grad_()
    x, y = _definition(case, v)
    total = (y * s["dy"].double()).sum()
    if case["branch"]:
        total = total + (x * s["dx_out"].double()).sum()
    asked = [k for k in _INPUTS if v[k] is not None]
    grads = dict(zip(asked, torch.autograd.grad(total, [v[k] for k in asked])))
    return {k: grads.get(k) for k in _INPUTS}


def _exact_linear(case, s):
    def values(c):
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        return torch.cat([table, -table])[c.long()]

    M, N, K = case["rows"], case["n"], case["k"]
    y = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for c in range(0, K, 2048):
        cols = slice(c, min(K, c + 2048))
        if case["format"] == "fp8r":
            y += s["xq"][:, cols].view(torch.float8_e4m3fn).double() @ s["w"][:, cols].view(
                torch.float8_e4m3fn).double().t()
            continue
        parts = []
        for q, b in ((s["xq"], s["x_scale"]), (s["w"], s["w_scale"])):
            q = q[:, cols.start // 2:cols.stop // 2]
            full = torch.empty(q.shape[0], cols.stop - cols.start, dtype=torch.float64, device="cuda")
            full[:, 0::2], full[:, 1::2] = values(q % 16), values(q // 16)
            b = b[:, cols.start // 16:cols.stop // 16].view(torch.float8_e4m3fn).double()
            parts.append(full * b.repeat_interleave(16, 1))
        y += parts[0] @ parts[1].t()
    if case["format"] == "fp8r":
        y = y * torch.outer(s["x_scale"].double(), s["w_scale"].double())
    else:
        y = y * s["input_scale"].double() * s["w_scale2"].double()
    y += s["bias"].double()
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    if case["act"] == "gelu_tanh":
        y = torch.nn.functional.gelu(y, approximate="tanh")
    if case["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    if case["gate"]:
        for g, rows in enumerate(_slices(case)):
            y[rows] *= s["gate"][g].double()
    if case["residual"]:
        y += s["residual"].double()
    return y
