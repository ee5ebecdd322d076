"""Cases, plain forms and exact values of the token-serving operators: rotary positions, appending
keys and values to a paged 8-bit cache, attention over that cache, and few-token products with
4-bit group-scaled weights.

own = False: run() computes the operators with elementary torch operations in 32 bits;
own = True:  run() makes the calls of block_scaled_precision_row_amd._lib.

The cache: K pages [pages, kv_heads, page, dim] and V pages [pages, kv_heads, dim, page] of E4M3
codes, and a power-of-two fp32 scale for each page and head of each. Page 0 is the pool's spare page
and belongs to no sequence.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3_MAX = 448.0


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # one decode step of a small batch: rotate the queries and keys of 48 far positions
        _rope("rope_step", 48, 40, 128, 128, "half", "plain", 100_000, "bf16", False),
        # a prompt's queries and keys, rotating half of each head, frequencies stretched for long contexts
        _rope("rope_prompt", 8192, 40, 128, 64, "interleaved", "yarn", 1_000_000, "fp16", False),
        # the gradient of the rotation, held in fp32
        _rope("rope_grad", 5001, 24, 64, 64, "half", "linear", 30_000, "fp32", True),
        # one decode step of a large batch: a token's keys and values for each sequence, queries rotated along
        _cache("append_step", "append", 96, 1, 1000, 32, 8, 128, 64, "bf16", rot=128, layout="half"),
        # prompts of several sequences appended at once, small pages, some sequences continued
        _cache("append_prompt", "append", 6, 2000, 300, 32, 8, 128, 16, "fp16", rot=64, layout="interleaved"),
        # one token of one short sequence: latency
        _cache("attention_one", "attention", 1, 1, 776, 32, 8, 128, 16, "bf16"),
        # one decode step of a ragged batch
        _cache("attention_batch", "attention", 64, 1, 8000, 32, 8, 128, 64, "bf16"),
        # one decode step of two long sequences with many queries to a key head
        _cache("attention_long", "attention", 2, 1, 130_000, 16, 2, 128, 128, "fp16"),
        # a chunk of prompt tokens of several sequences over what they have cached
        _cache("attention_prompt", "attention", 3, 1500, 4500, 32, 8, 128, 64, "bf16"),
        # one token through a small projection: latency
        _int4("int4_one", 1, 4096, 4096, 128, False, "bf16"),
        # one token through a wide projection with zero points
        _int4("int4_wide", 1, 16384, 8192, 64, True, "bf16"),
        # a few tokens (a decode batch) through a projection with small groups
        _int4("int4_few", 24, 12288, 4096, 32, True, "fp16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "append", "attention", "attention", "int4"])
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        return _rope(None, spread(1, 4000), rng.randint(1, 40), dim, rng.choice([dim, dim // 2, dim // 4]),
                     rng.choice(["half", "interleaved"]), rng.choice(["plain", "linear", "yarn"]),
                     spread(100, 1_000_000), rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.4)
    if op == "int4":
        group = rng.choice([32, 64, 128])
        return _int4(None, spread(1, 48), spread(64, 1000) * rng.choice([1, 8]), 128 * spread(2, 64), group,
                     rng.random() < 0.5, rng.choice(["bf16", "fp16"]))
    dim, kv = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 4, 8])
    heads, page, kind = kv * rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "fp16"])
    if op == "append":
        return _cache(None, op, rng.randint(1, 40), rng.choice([1, 1, spread(2, 300)]), spread(1, 1000), heads, kv, dim,
                      page, kind, rot=rng.choice([0, dim, dim // 2]), layout=rng.choice(["half", "interleaved"]))
    new, window = rng.choice([1, 1, 1, spread(2, 600)]), rng.choice([0, 0, spread(16, 2000)])
    if new == 1:
        return _cache(None, op, rng.randint(1, 16), new, spread(1, 8000), heads, kv, dim, page, kind, window=window)
    return _cache(None, op, rng.randint(1, 3), new, spread(1, 3000), min(heads, 4 * kv), kv, dim, page, kind,
                  window=window)


def _named(name, case):
    return dict(case, name=name) if name else case


def _rope(name, tokens, heads, dim, rot, layout, scaling, far, kind, backward):
    return _named(name, {"op": "rope", "tokens": tokens, "heads": heads, "dim": dim, "rot": rot, "layout": layout,
                         "scaling": scaling, "far": far, "type": kind, "backward": backward})


def _cache(name, op, seqs, new, past, heads, kv_heads, dim, page, kind, rot=0, layout="half", window=0):
    """`new`: the most new tokens of a sequence (1: one each), `past`: the most that a sequence has cached."""
    case = {"op": op, "seqs": seqs, "new": new, "past": past, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": page, "type": kind}
    case.update({"rot": rot, "layout": layout} if op == "append" else {"window": window})
    return _named(name, case)


def _int4(name, tokens, n, k, group, zeros, kind):
    return _named(name, {"op": "int4", "tokens": tokens, "n": n, "k": k, "group": group, "zeros": zeros, "type": kind})


# ---- inputs --------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    return {"rope": _prepare_rope, "append": _prepare_cache, "attention": _prepare_cache,
            "int4": _prepare_int4}[case["op"]](case, seed, g, state)


def _frequencies(rot, scaling):
    """Inverse frequencies fp32 [rot / 2] and the factor of cos and sin, as a model's configuration gives them."""
    base, factor, trained = 500_000.0, 8.0, 8192
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        turns = trained * f / (2 * math.pi)  # turns over the trained length: many stay, few are stretched
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    return f.float(), scale


def _prepare_rope(case, seed, g, state):
    x = torch.randn(case["tokens"], case["heads"], case["dim"], generator=g, device="cuda").to(TYPES[case["type"]])
    positions = torch.randint(0, case["far"], (case["tokens"],), generator=g, device="cuda")
    f, scale = _frequencies(case["rot"], case["scaling"])
    state.update(x=x, positions=positions, inv_freq=f.cuda(), factor=scale, y=torch.empty_like(x))
    return state


def _lengths(case):
    """New and cached tokens of each sequence: the case's own, so that outputs of all inputs have one shape."""
    g = torch.Generator()
    g.manual_seed(1000 * case["seqs"] + case["past"] + case["new"])
    B = case["seqs"]
    new = torch.ones(B, dtype=torch.int64)
    if case["new"] > 1:
        new = torch.randint(max(1, case["new"] // 2), case["new"] + 1, (B,), generator=g)
    return new, torch.randint(case["past"] // 2, case["past"] + 1, (B,), generator=g)


def _prepare_cache(case, seed, g, state):
    B, page, dim, kv, kind = case["seqs"], case["page"], case["dim"], case["kv_heads"], TYPES[case["type"]]
    new, past = _lengths(case)
    lens = past + new
    cg = torch.Generator()
    cg.manual_seed(seed)
    pages = (lens + page - 1) // page
    width, total = int(pages.max()), int(pages.sum()) + 1
    order = torch.randperm(total - 1, generator=cg) + 1
    table = torch.full((B, width), -1, dtype=torch.int32)
    first = 0
    for b in range(B):
        n = int(pages[b])
        table[b, :n] = order[first:first + n]
        first += n
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    T = int(cu[-1])

    def codes(shape):
        return (torch.randn(shape, generator=g, device="cuda") * 60).clamp(-E4M3_MAX, E4M3_MAX).to(
            torch.float8_e4m3fn).view(torch.uint8)

    def scales():
        return torch.exp2(torch.randint(-7, -4, (total, kv), generator=g, device="cuda").float())

    qkv = torch.randn(T, case["heads"] + 2 * kv, dim, generator=g, device="cuda").to(kind)
    state.update(
        q=qkv[:, :case["heads"]], k=qkv[:, case["heads"]:case["heads"] + kv], v=qkv[:, case["heads"] + kv:],
        cu=cu.int().cuda(), lens=lens.int().cuda(), table=table.cuda(), most=int(new.max()),
        k_cache=codes((total, kv, page, dim)), v_cache=codes((total, kv, dim, page)), k_scale=scales(),
        v_scale=scales(), y=torch.empty(T, case["heads"], dim, dtype=kind, device="cuda"))
    if case["op"] == "append":
        f, scale = _frequencies(case["rot"], "yarn") if case["rot"] else (None, 1.0)
        state.update(inv_freq=f.cuda() if case["rot"] else None, factor=scale)
    else:
        state.update(lse=torch.empty(T, case["heads"], device="cuda"), scale=dim ** -0.5)
    return state


def _prepare_int4(case, seed, g, state):
    M, N, K, groups, kind = case["tokens"], case["n"], case["k"], case["k"] // case["group"], TYPES[case["type"]]
    state.update(
        x=torch.randn(M, K, generator=g, device="cuda").to(kind),
        w=torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
        w_scale=(torch.rand(N, groups, generator=g, device="cuda") * 0.004 + 0.001).to(kind),
        w_zero=torch.randint(4, 12, (N, groups), generator=g, device="cuda", dtype=torch.uint8)
        if case["zeros"] else None,
        y=torch.empty(M, N, dtype=kind, device="cuda"))
    return state


# ---- one pass ------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention,
            "int4": _plain_int4}[case["op"]](case, state)


def _own(case, s):
    from block_scaled_precision_row_amd import _lib as L
    layout = L.BSQ_ROPE_INTERLEAVED if case.get("layout") == "interleaved" else L.BSQ_ROPE_HALF
    if case["op"] == "rope":
        return L.bsq_rope(s["x"], s["positions"], s["inv_freq"], layout, s["factor"], backward=case["backward"], y=s["y"])
    if case["op"] == "append":
        L.bsq_kv_append(s["k"], s["v"], s["cu"], s["lens"], s["table"], s["k_cache"], s["v_cache"], s["k_scale"],
                        s["v_scale"], inv_freq=s["inv_freq"], layout=layout, attn_factor=s["factor"], q=s["q"],
                        q_out=s["y"])
        return _appended(s, s["y"])
    if case["op"] == "attention":
        y, lse = L.bsq_attention_kv8(s["q"], s["cu"], s["lens"], s["table"], s["k_cache"], s["v_cache"], s["k_scale"],
                                     s["v_scale"], s["most"], softmax_scale=s["scale"], window=case["window"],
                                     y=s["y"], lse=s["lse"])
        return {"y": y, "lse": lse}
    return L.bsq_gemm_int4g(s["x"], s["w"], s["w_scale"], s["w_zero"], y=s["y"])


def _appended(s, q):
    return {"k": s["k_cache"].view(torch.float8_e4m3fn), "v": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"], "q": q}


def _rotate(x, positions, inv_freq, layout, factor, backward):
    """x [T, H, D] as fp32 with its first 2 * len(inv_freq) dims rotated; the angles in 64 bits."""
    rot = 2 * inv_freq.numel()
    angle = positions.double()[:, None, None] * inv_freq.double()
    cos = (angle.cos() * factor).float()
    sin = (angle.sin() * (-factor if backward else factor)).float()
    x = x.float()
    r = x[..., :rot]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_rope(case, s):
    y = _rotate(s["x"], s["positions"], s["inv_freq"], case["layout"], s["factor"], case["backward"])
    s["y"].copy_(y)
    return s["y"]


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _encode(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _place(s, tokens):
    """Sequence and place in it of each of the tokens."""
    t = torch.arange(tokens, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    return b, t - s["cu"][b]


def _plain_append(case, s):
    page, cu, lens, T = case["page"], s["cu"].long(), s["lens"].long(), s["k"].shape[0]
    n = cu[1:] - cu[:-1]
    past = lens - n
    q, k = s["q"], s["k"]
    if case["rot"]:
        b, i = _place(s, T)
        at = past[b] + i
        q = _rotate(q, at, s["inv_freq"], case["layout"], s["factor"], False)
        k = _rotate(k, at, s["inv_freq"], case["layout"], s["factor"], False)
    s["y"].copy_(q)
    # every page that a sequence's new tokens touch, [B, touched]; the others stand for the spare page 0
    touched = (s["most"] + page - 2) // page + 1
    at = past[:, None] // page + torch.arange(touched, device="cuda")
    live = (at * page < lens[:, None]) & (n[:, None] > 0)
    ids = torch.where(live, s["table"].gather(1, at.clamp(max=s["table"].shape[1] - 1)).long(), 0).flatten()
    i = at[:, :, None] * page + torch.arange(page, device="cuda") - past[:, None, None]
    is_new = ((i >= 0) & (i < n[:, None, None]) & live[:, :, None]).flatten(0, 1)
    is_old = ((i < 0) & live[:, :, None]).flatten(0, 1)
    source = (cu[:-1, None, None] + i).clamp(0, T - 1).flatten(0, 1)
    for x, cache, scale, swap in ((k, s["k_cache"], s["k_scale"], False), (s["v"], s["v_cache"], s["v_scale"], True)):
        x = x.float()[source].transpose(1, 2)  # [pages, heads, page, dim]
        x = torch.where(is_new[:, None, :, None], x, 0.0)
        m, e = torch.frexp(x.abs().amax((2, 3)))
        fresh = torch.where(m > 0, torch.exp2((e - 9 + (m > 0.875).int()).float()), 0.0)
        before = torch.where(is_old.any(1)[:, None], scale[ids], 0.0)
        after = torch.where(is_new.any(1)[:, None], torch.maximum(before, fresh), scale[ids])
        ratio = torch.where(after > 0, before / after, 0.0)
        put = torch.where(after > 0, 1 / after, 0.0)
        old = cache[ids].transpose(2, 3) if swap else cache[ids]
        kept = torch.where(is_old[:, None, :, None], _encode(_decode(old.contiguous()) * ratio[:, :, None, None]), old)
        out = torch.where(is_new[:, None, :, None], _encode(x * put[:, :, None, None]), kept)
        cache[ids] = out.transpose(2, 3) if swap else out
        scale[ids] = after
    return _appended(s, s["y"])


def _plain_attention(case, s):
    kv, dim, page, most = case["kv_heads"], case["dim"], case["page"], s["most"]
    T, group = s["q"].shape[0], case["heads"] // kv
    cu, lens, ids = s["cu"].long(), s["lens"].long(), s["table"].clamp(min=0).long()
    n = cu[1:] - cu[:-1]
    B, tokens = ids.shape[0], ids.shape[1] * page
    k = _decode(s["k_cache"][ids]) * s["k_scale"][ids][..., None, None]   # [B, pages, kv, page, dim]
    k = k.permute(0, 2, 4, 1, 3).reshape(B * kv, dim, tokens)
    v = _decode(s["v_cache"][ids]) * s["v_scale"][ids][..., None, None]   # [B, pages, kv, dim, page]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, kv, tokens, dim)
    at = torch.arange(tokens, device="cuda")
    v = torch.where((at < lens[:, None])[:, None, :, None], v, 0.0).reshape(B * kv, tokens, dim)
    i = torch.arange(most, device="cuda")
    q = s["q"][(cu[:-1, None] + i).clamp(max=T - 1)].float()              # [B, most, heads, dim]
    q = q.view(B, most, kv, group, dim).permute(0, 2, 1, 3, 4).reshape(B * kv, most * group, dim)
    place = (lens - n)[:, None] + i                                       # [B, most]
    seen = (at <= place[..., None]) & (at < lens[:, None, None])
    if case["window"]:
        seen = seen & (at > place[..., None] - case["window"])
    seen = seen[:, None, :, None, :].expand(B, kv, most, group, tokens).reshape(B * kv, most * group, tokens)
    w = torch.bmm(q, k) * s["scale"]
    w = w.masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top.isfinite(), top, 0.0)).exp_()
    total = w.sum(-1, keepdim=True)
    y = torch.where(total > 0, torch.bmm(w, v) / total, 0.0).view(B, kv, most, group, dim)
    lse = (top + total.log()).view(B, kv, most, group)
    b, i = _place(s, T)
    s["y"].copy_(y.permute(0, 2, 1, 3, 4).reshape(B, most, -1, dim)[b, i])
    s["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(B, most, -1)[b, i])
    return {"y": s["y"], "lse": s["lse"]}


def _plain_int4(case, s):
    w = torch.stack([s["w"] & 15, s["w"] >> 4], -1).view(case["n"], -1, case["group"]).float()
    w = (w - (8.0 if s["w_zero"] is None else s["w_zero"].float()[..., None])) * s["w_scale"].float()[..., None]
    s["y"].copy_(s["x"].float() @ w.view(case["n"], case["k"]).t())
    return s["y"]


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["type"]]
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 2 * n * size + 8 * case["tokens"], "flops": 3 * n * case["rot"] // case["dim"]}
    if case["op"] == "int4":
        weights = case["n"] * case["k"]
        scales = weights // case["group"] * (size + (1 if case["zeros"] else 0))
        return {"bytes": weights // 2 + scales + size * case["tokens"] * (case["k"] + case["n"]),
                "flops": 2 * case["tokens"] * weights}
    new, past = _lengths(case)
    rows = int(new.sum())
    if case["op"] == "append":
        values = rows * case["kv_heads"] * case["dim"]
        return {"bytes": 2 * values * (size + 1) + 2 * size * rows * case["heads"] * case["dim"],
                "flops": 3 * (rows * case["heads"] * case["dim"] + values)}
    window = case["window"] or 1 << 40
    kept = int(torch.minimum(past + new, window + new - 1).sum())  # tokens that some row sees
    seen = sum(min(p + i + 1, window) for p, n in zip(past.tolist(), new.tolist()) for i in range(n))
    return {"bytes": 2 * kept * case["kv_heads"] * case["dim"] + rows * case["heads"] * (2 * size * case["dim"] + 4),
            "flops": 4 * seen * case["heads"] * case["dim"]}


# ---- exact values, from the definitions, in 64 bits ----------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(s["x"], s["positions"], s["inv_freq"], case["layout"], s["factor"],
                               -1.0 if case["backward"] else 1.0)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "attention":
        return _exact_attention(case, s)
    K = case["k"]
    y = torch.zeros(case["tokens"], case["n"], dtype=torch.float64, device="cuda")
    for c in range(0, K, case["group"]):  # y = sum over groups of scale * (x . codes - zero * sum x)
        xs = s["x"][:, c:c + case["group"]].double()
        pair = s["w"][:, c // 2:(c + case["group"]) // 2].int()
        dots = xs[:, 0::2] @ (pair % 16).double().t() + xs[:, 1::2] @ (pair // 16).double().t()
        zero = 8.0 if s["w_zero"] is None else s["w_zero"][:, c // case["group"]].double()
        y += s["w_scale"][:, c // case["group"]].double() * (dots - xs.sum(1, keepdim=True) * zero)
    return y


def _exact_rotation(x, positions, inv_freq, layout, factor, sign):
    pairs = inv_freq.numel()
    y = x.double().clone()
    z = torch.view_as_complex(torch.stack(
        [y[..., :pairs], y[..., pairs:2 * pairs]] if layout == "half"
        else [y[..., :2 * pairs:2], y[..., 1:2 * pairs:2]], -1).contiguous())
    turn = torch.polar(torch.full_like(inv_freq, factor, dtype=torch.float64)[None].expand(len(positions), -1),
                       sign * torch.outer(positions.double(), inv_freq.double()))
    z = z * turn[:, None, :]
    if layout == "half":
        y[..., :pairs], y[..., pairs:2 * pairs] = z.real, z.imag
    else:
        y[..., :2 * pairs:2], y[..., 1:2 * pairs:2] = z.real, z.imag
    return y


def _nearest_e4m3(x):
    """The E4M3 value nearest to x (ties to even), in fp64: steps of an eighth of x's power of two, at least 2^-9."""
    power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(power - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(case, s):
    page, cu, lens = case["page"], s["cu"].tolist(), s["lens"].tolist()
    k_cache = s["k_cache"].view(torch.float8_e4m3fn).double()
    v_cache = s["v_cache"].view(torch.float8_e4m3fn).double().transpose(2, 3).contiguous()
    k_scale, v_scale = s["k_scale"].double(), s["v_scale"].double()
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if case["rot"]:
        at = torch.cat([torch.arange(n - (e - c), n) for c, e, n in zip(cu[:-1], cu[1:], lens)]).cuda()
        q = _exact_rotation(q, at, s["inv_freq"], case["layout"], s["factor"], 1.0)
        k = _exact_rotation(k, at, s["inv_freq"], case["layout"], s["factor"], 1.0)
    table = s["table"].tolist()
    for b, n in enumerate(lens):
        start = n - (cu[b + 1] - cu[b])
        for p in range(start // page, (n + page - 1) // page):
            lo, hi = max(start, p * page), min(n, (p + 1) * page)
            rows, first, at = slice(cu[b] + lo - start, cu[b] + hi - start), lo - p * page, table[b][p]
            for x, cache, scale in ((k, k_cache, k_scale), (v, v_cache, v_scale)):
                x = x[rows].transpose(0, 1)  # [heads, tokens, dim]
                most = x.abs().amax((1, 2))
                # the least power of two that brings the largest value within E4M3
                now = torch.exp2(torch.ceil(torch.log2(most / E4M3_MAX)))
                if first:
                    now = torch.maximum(now, scale[at])
                    cache[at, :, :first] = _nearest_e4m3(cache[at, :, :first] * (scale[at] / now)[:, None, None])
                cache[at, :, first:first + hi - lo] = _nearest_e4m3(x / now[:, None, None])
                scale[at] = now
    return {"k": k_cache, "v": v_cache.transpose(2, 3).contiguous(), "k_scale": k_scale, "v_scale": v_scale, "q": q}


def _exact_attention(case, s):
    kv, dim, page, group = case["kv_heads"], case["dim"], case["page"], case["heads"] // case["kv_heads"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        ids = s["table"][b, :(n + page - 1) // page].long()
        rows = slice(cu[b], cu[b + 1])
        place = torch.arange(n - (cu[b + 1] - cu[b]), n, device="cuda")[:, None]
        at = torch.arange(n, device="cuda")
        hidden = (at > place) if not case["window"] else (at > place) | (at <= place - case["window"])
        for h in range(kv):
            k = (s["k_cache"][ids, h].view(torch.float8_e4m3fn).double() * s["k_scale"][ids, h].double()[:, None, None])
            k = k.reshape(-1, dim)[:n]
            v = (s["v_cache"][ids, h].view(torch.float8_e4m3fn).double() * s["v_scale"][ids, h].double()[:, None, None])
            v = v.transpose(1, 2).reshape(-1, dim)[:n]
            for j in range(h * group, (h + 1) * group):
                w = (s["q"][rows, j].double() @ k.t()) * s["scale"]
                w[hidden] = -math.inf
                lse[rows, j] = torch.logsumexp(w, -1)
                y[rows, j] = torch.softmax(w, -1) @ v
    return {"y": y, "lse": lse}
