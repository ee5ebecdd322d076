"""A block of a diffusion transformer run with the operators as they are used together: norm, scale and shift into codes,
a linear with bias, rotary positions of rows and columns, attention (plain, in fp32 on the CPU), a linear into the gated
residual, norm again, a linear with activation and one into the gated residual, for images of several sizes packed.
Every stage is held to the oracle on what the stage before it gave."""
import numpy as np
import pytest
import torch

from oracle import block
from oracle.codec import e2m1_decode, e4m3_decode
from tests.block_util import f64, forward_bounds, rounded
from tests.test_gpu_epilogue import check, product_bound
from tests.test_gpu_rope_axes import bound

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L

D, HEADS, DIM, INNER = 512, 8, 64, 1280
SIZES = [(9, 13), (16, 16), (5, 3)]          # rows and columns of each image
EPS = 1e-6


class Linear:
    """A weight in one of the formats, with the fp64 values it stands for, and the calls that take it."""

    def __init__(self, fmt, n, k, g):
        self.fmt = fmt
        w = (torch.randn(n, k, generator=g) / k ** 0.5).bfloat16().cuda()
        self.bias = (torch.randn(n, generator=g) * 0.2).bfloat16().cuda()
        if fmt == "fp8r":
            self.w = L.bsq_quantize_act_fp8r(w)
            self.value = e4m3_decode(self.w[0].cpu().numpy()).astype(np.float64) * f64(self.w[1])[:, None]
            self.input_scale = None
        else:
            s2 = L.bsq_calibrate_global_scale(w)
            self.w = (*L.bsq_quantize_act_nvfp4(w, s2), s2)
            self.value = self._nvfp4(self.w[0], self.w[1], s2)
            self.input_scale = torch.tensor([8.0 / (6 * 448)], device="cuda")

    @staticmethod
    def _nvfp4(codes, scales, s2):
        c = codes.cpu().numpy()
        v = np.stack([e2m1_decode(c & 15), e2m1_decode(c >> 4)], -1).reshape(len(c), -1).astype(np.float64)
        return v * np.repeat(e4m3_decode(scales.cpu().numpy()).astype(np.float64), 16, 1) * float(s2)

    def encode(self, x):
        return L.bsq_quantize_act_fp8r(x) if self.fmt == "fp8r" else L.bsq_quantize_act_nvfp4(x, self.input_scale)

    def norm(self, x, **kw):
        y, s, out = L.bsq_block_norm(x, L.BSQ_NORM_LAYER, EPS, y_global=self.input_scale,
                                     out_format=L.BSQ_FMT_FP8R if self.fmt == "fp8r" else L.BSQ_FMT_NVFP4, **kw)
        return (y, s), out

    def decoded(self, q):
        if self.fmt == "fp8r":
            return e4m3_decode(q[0].cpu().numpy()).astype(np.float64) * f64(q[1])[:, None]
        return self._nvfp4(q[0], q[1], self.input_scale)

    def __call__(self, q, **kw):
        if self.fmt == "fp8r":
            return L.bsq_gemm_fp8r_q_epilogue(*q, *self.w, bias=self.bias, **kw)
        return L.bsq_gemm_nvfp4_q_epilogue(*q, self.input_scale, *self.w, bias=self.bias, **kw)


def attention(q, k, v, starts):
    out = torch.empty_like(q, dtype=torch.float32)
    for a, b in zip(starts[:-1], starts[1:]):
        s = torch.softmax(torch.einsum("thd,shd->hts", q[a:b].float(), k[a:b].float()) * DIM ** -0.5, -1)
        out[a:b] = torch.einsum("hts,shd->thd", s, v[a:b].float())
    return out.flatten(1).bfloat16()


@pytest.mark.parametrize("fmt", ["fp8r", "nvfp4"])
def test_block(fmt):
    g = torch.Generator().manual_seed(0)
    n = [r * c for r, c in SIZES]
    starts = [0, *np.cumsum(n).tolist()]
    T = starts[-1] + 7                                            # and rows behind the last image
    group = block.group_of_rows(T, len(n), starts)
    live = group >= 0
    st = torch.tensor(starts, dtype=torch.int32).cuda()
    x = torch.randn(T, D, generator=g).bfloat16().cuda()
    mod = (torch.randn(len(n), 6 * D, generator=g) * 0.3).bfloat16().cuda()
    scale1, shift1, gate1, scale2, shift2, gate2 = mod.split(D, 1)
    pos = torch.zeros(T, 2, dtype=torch.int64)
    for a, (r, c) in zip(starts, SIZES):
        pos[a:a + r * c] = torch.stack(torch.meshgrid(torch.arange(r), torch.arange(c), indexing="ij"), -1).view(-1, 2)
    inv = torch.cat([L.bsq_rope_inv_freq(DIM // 2, 10000.0)[0]] * 2)
    qkv, out, up, down = (Linear(fmt, *s, g) for s in ((3 * D, D), (D, D), (INNER, D), (D, INNER)))
    start = x.clone()

    def product(layer, codes):
        a = layer.decoded(codes)
        return a @ layer.value.T, product_bound(fmt, a.shape[1], np.abs(a) @ np.abs(layer.value).T)

    def check_codes(layer, codes, x, scale, shift):
        _, _, y, ey = forward_bounds(f64(x), "layer", EPS, group, scale=f64(scale), shift=f64(shift))
        got, y, ey = layer.decoded(codes)[live], y[live], ey[live]
        if fmt == "fp8r":
            d = f64(codes[1])[live][:, None]
            assert np.all(np.abs(got - y) <= (2.0 ** -4 + 2.0 ** -20) * np.abs(y) + 2.0 ** -10 * d + 1.1 * ey + 1.1 * ey.max(-1, keepdims=True))
        else:
            unit = np.repeat(e4m3_decode(codes[1].cpu().numpy()).astype(np.float64)[live], 16, 1) * float(layer.input_scale)
            tiny = 2.0 ** -9 * 6 * float(layer.input_scale)
            assert np.all(np.abs(got - y) <= np.maximum(0.25 * unit, np.abs(y) / 4) * (1 + 2.0 ** -20) + 2 * tiny + 1.1 * ey)

    codes, _ = qkv.norm(x, scale=scale1, shift=shift1, starts=st)
    check_codes(qkv, codes, x, scale1, shift1)
    codes[0][~torch.from_numpy(live)] = 0                         # (rows of no image: whatever the buffer held)
    if fmt == "fp8r":
        codes[1][~torch.from_numpy(live)] = 0
    h = qkv(codes)
    check(h, *product(qkv, codes), qkv.bias, "none", None, None, None)
    heads = h.view(T, 3 * HEADS, DIM)
    q0 = heads[:, :2 * HEADS].cpu()
    L.bsq_rope_axes(heads[:, :2 * HEADS], pos.cuda(), inv.cuda(), [DIM // 4, DIM // 4], y=heads[:, :2 * HEADS])
    ref = block.rope_axes(f64(q0), pos.numpy(), f64(inv), [DIM // 4, DIM // 4])
    assert np.all(np.abs(f64(heads[:, :2 * HEADS]) - ref) <= bound(q0, ref, DIM // 2, 1.0, "bf16", False))
    q, k, v = heads.cpu().split(HEADS, 1)
    a = attention(q[:starts[-1]], k[:starts[-1]], v[:starts[-1]], starts)
    a = torch.cat([a, torch.zeros(7, D, dtype=torch.bfloat16)]).cuda()

    codes = out.encode(a)
    before = x.clone()
    assert out(codes, gate=gate1, residual=x, starts=st, y=x) is x   # the stream, in place
    check(x, *product(out, codes), out.bias, "none", gate1, before, group)
    # the same by the norm's own gated residual: the branch rounded on its way
    branch = out(codes)
    (codes2, _), (codes3, other) = up.norm(x, scale=scale2, shift=shift2, starts=st), up.norm(
        before, branch=branch, gate=gate1, scale=scale2, shift=shift2, starts=st)
    want = f64(before) + block._rows(f64(gate1), group, 0.0, D) * f64(branch)
    assert np.all(np.abs(f64(other) - want)[live] <= (2.0 ** -20 * np.abs(want) + rounded(want, torch.bfloat16) + 2.0 ** -22)[live])
    slack = 2.0 ** -8 * np.abs(block._rows(f64(gate1), group, 0.0, D) * f64(branch)) + 2.0 ** -7 * np.abs(f64(x)) + 2.0 ** -18
    assert np.all(np.abs(f64(other) - f64(x))[live] <= slack[live])
    check_codes(up, codes2, x, scale2, shift2)
    codes2[0][~torch.from_numpy(live)] = 0
    if fmt == "fp8r":
        codes2[1][~torch.from_numpy(live)] = 0
    m = up(codes2, act=L.BSQ_ACT_GELU_TANH)
    check(m, *product(up, codes2), up.bias, "gelu_tanh", None, None, None)
    codes = down.encode(m)
    before = x.clone()
    down(codes, gate=gate2, residual=x, starts=st, y=x)
    check(x, *product(down, codes), down.bias, "none", gate2, before, group)
    assert torch.equal(x[starts[-1]:], start[starts[-1]:])


@pytest.mark.parametrize("fmt", ["fp8r", "nvfp4"])
def test_block_captured(fmt):
    """The block but for its attention, captured and replayed with other rows and images: the eager run's bits."""
    g = torch.Generator().manual_seed(1)
    T = 300
    x = torch.randn(T, D, generator=g).bfloat16().cuda()
    st = torch.tensor([0, 100, 180, T], dtype=torch.int32).cuda()
    mod = (torch.randn(3, 3 * D, generator=g) * 0.3).bfloat16().cuda()
    scale, shift, gate = mod.split(D, 1)
    pos, inv = torch.randint(0, 40, (T, 2)).cuda(), torch.cat([L.bsq_rope_inv_freq(DIM // 2, 10000.0)[0]] * 2).cuda()
    qk, up, down = (Linear(fmt, *s, g) for s in ((D, D), (INNER, D), (D, INNER)))

    def run():
        codes, _ = up.norm(x, scale=scale, shift=shift, starts=st)
        heads = qk(codes).view(T, HEADS, DIM)
        r = L.bsq_rope_axes(heads, pos, inv, [DIM // 4, DIM // 4])
        m = up(codes, act=L.BSQ_ACT_SILU)
        return [codes[0], r, m, down(down.encode(m), gate=gate, residual=x, starts=st)]

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i in range(4):
        x.normal_()
        mod.normal_(0, 0.3)
        pos.random_(0, 99)
        st.copy_(torch.tensor([0, 20 * i, 200 + i, T]))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
