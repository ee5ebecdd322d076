"""GPU test of the cache's operators between the block-scaled linears: an nvfp4 projection to queries, keys and values,
append, attention, and an fp8r projection back, a prompt and steps of two sequences, eagerly and replayed from a graph."""
import numpy as np
import pytest
import torch

from oracle import quant, serve
from tests.serve_util import Cache, attention_bounds, f64, gpu, starts

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L
    from block_scaled_precision_row_amd import synthetic as syn

H, HQ, D, K = 2, 8, 64, 256


def bf16(bits):
    return gpu(bits.view(np.int16)).view(torch.bfloat16)


def weights():
    w1, w2 = syn.weights(syn.TINY, (HQ + 2 * H) * D, K), syn.weights(syn.TINY, K, HQ * D)
    g = quant.calibrate_global_scale(w1)
    wq, sf = quant.quantize_nvfp4(w1, g)
    w8, s8 = quant.quantize_fp8r(w2)
    return gpu(wq), gpu(sf), torch.tensor([float(g)], device="cuda"), gpu(w8), gpu(s8), L.bsq_rope_inv_freq(D, 10000.0)[0].cuda()


def layer(w, x, cu, lens, table, pools, most, ws=None):
    wq, sf, g, w8, s8, freq = w
    qkv = L.bsq_gemm_nvfp4(x, wq, sf, g, flags=L.BSQ_WEIGHT_ONLY).view(-1, HQ + 2 * H, D)
    L.bsq_kv_append(qkv[:, HQ:HQ + H], qkv[:, HQ + H:], cu, lens, table, *pools, freq, q=qkv[:, :HQ], q_out=qkv[:, :HQ])
    y, _ = L.bsq_attention_kv8(qkv[:, :HQ], cu, lens, table, *pools, most, workspace=ws)
    return qkv, y, L.bsq_gemm_fp8r(y.view(-1, HQ * D), w8, s8)


def test_a_layer_of_block_scaled_linears():
    w, c = weights(), Cache(5, [44, 27], H, D, 16)
    table, pools = gpu(c.table), [gpu(a) for a in (c.kc, c.vc, c.ks, c.vs)]
    lens = np.zeros(2, np.int32)
    for rows in ([40, 23], [1, 1], [1, 1]):
        lens = (lens + rows).astype(np.int32)
        cu = starts(rows)
        x = bf16(syn.activations(syn.TINY, int(cu[-1]), K))
        qkv, y, out = layer(w, x, gpu(cu), gpu(lens), table, pools, max(rows))
        ref, _, parts = serve.attention(f64(qkv)[:, :HQ], cu, lens, c.table, *(p.cpu().numpy() for p in pools), D ** -0.5)
        assert np.all(np.abs(f64(y) - ref) <= attention_bounds(ref, np.zeros(ref.shape[:2]), parts, torch.bfloat16, D)[0])
        # the projections are what they are alone
        assert torch.equal(out, L.bsq_gemm_fp8r(y.reshape(-1, HQ * D).clone(), w[3], w[4]))
        plain = L.bsq_gemm_nvfp4(x, *w[:3], flags=L.BSQ_WEIGHT_ONLY).view(-1, HQ + 2 * H, D)
        pos = np.concatenate([np.arange(n - r, n) for n, r in zip(lens, rows)])
        assert torch.equal(qkv[:, HQ + H:], plain[:, HQ + H:])
        assert torch.equal(qkv[:, :HQ], L.bsq_rope(plain[:, :HQ], gpu(pos), w[5]))


def test_its_step_replays():
    w, c = weights(), Cache(6, [60, 50], H, D, 16)
    table, cu = gpu(c.table), gpu(starts([1, 1]))
    pools, other = ([gpu(a) for a in (c.kc, c.vc, c.ks, c.vs)] for _ in range(2))
    lens = torch.tensor([20, 30], dtype=torch.int32, device="cuda")
    x = bf16(syn.activations(syn.TINY, 2, K))
    ws = torch.empty(max(L.bsq_attention_kv8_workspace_bytes(2, 2, 1, HQ, H, D), 256), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(w, x, cu, lens, table, pools, 1, ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, y, out = layer(w, x, cu, lens, table, pools, 1, ws)
    for i in range(4):
        x.copy_(bf16(syn.activations(syn.TINY, 2 + i, K))[-2:])
        lens.add_(torch.tensor([2, 1 + i], dtype=torch.int32, device="cuda"))
        for a, b in zip(other, pools):
            a.copy_(b)
        graph.replay()
        _, ey, eager = layer(w, x, cu, lens, table, other, 1)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(y, ey) and all(torch.equal(a, b) for a, b in zip(pools, other))
