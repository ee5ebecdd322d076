"""GPU tests of rotations at far positions: angles p w in exact rational arithmetic, reduced by 2 pi to 100 digits. The
bounds are those of near positions (tests/serve_util.py): positions of any magnitude below 2^53 lose nothing."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import serve
from tests.serve_util import DTYPES, f64, gpu, starts, u

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679, 10 ** 100)
FAR = [0, 1, -3, 2 ** 24 + 7, 2 ** 31 - 1, 2 ** 33 + 12345, 2 ** 40 + 99, -(2 ** 45) - 31, 2 ** 50 + 1, 2 ** 52 + 3, 2 ** 53 - 1,
       -(2 ** 53) + 1]


def turns(positions, w):
    """Cosines and sines [T, pairs] of p w, the angle exact up to the last rounding."""
    out = np.zeros((len(positions), len(w)))
    units = [int(Fraction(float(f)) / (2 * PI) * 2 ** 260) for f in w]   # of a turn, 2^-260 each: 2^53 of them err by 2^-207
    for i, p in enumerate(positions):
        for j, f in enumerate(units):
            part = (int(p) * f) % 2 ** 260
            out[i, j] = float(Fraction(part - 2 ** 260 if part >= 2 ** 259 else part, 2 ** 260))
    return np.cos(2 * np.pi * out), np.sin(2 * np.pi * out)


def rotate(x, positions, w, interleaved, factor=1.0, backward=False):
    y, half = np.array(x, dtype=np.float64), len(w)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    c, s = turns(positions, w)
    c, s = (factor * c)[:, None], ((-factor if backward else factor) * s)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size = np.zeros(y.shape)
    size[..., a] = size[..., b] = factor * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, size


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved,backward", [(False, False), (True, True)])
@pytest.mark.parametrize("H,D,rot", [(2, 128, 128), (3, 66, 34), (40, 64, 32)])   # 34: the kernel for any rot and stride
def test_far_positions_lose_nothing(H, D, rot, interleaved, backward, kind):
    x = torch.from_numpy(np.random.default_rng(D).standard_normal((len(FAR), H, D))).to(DTYPES[kind])
    w, _ = L.bsq_rope_inv_freq(rot, 10000.0, L.BSQ_ROPE_NTK, 8.0)
    ref, size = rotate(f64(x), FAR, f64(w), interleaved, 1.25, backward)
    y = f64(L.bsq_rope(x.cuda(), gpu(np.array(FAR)), w.cuda(), L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF, 1.25,
                       backward=backward))
    bound = np.where(size > 0, u(DTYPES[kind]) * np.abs(ref) + 2.0 ** -21 * size + (2.0 ** -25 if kind == "fp16" else 0.0), 0.0)
    off = np.abs(y - ref)
    assert np.all(off <= bound), (off / (bound + 1e-300)).max(axis=(1, 2))


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_at_far_positions_bit_for_bit(kind, interleaved):
    """Two million keys of a sequence of 2^31 - 2000 tokens: the codes of the keys in 64 bits, all of them."""
    T, H, D, page, n = 4000, 4, 128, 256, 2 ** 31 - 2000
    first, width = (n - T) // page, (n - 1) // page + 1
    many = width - first
    table = np.full((1, width), -1, np.int32)
    table[0, first:] = np.random.default_rng(1).permutation(many)
    rng = np.random.default_rng(2)
    k, v = (torch.from_numpy(rng.standard_normal((T, H, D))).to(DTYPES[kind]) for _ in range(2))
    w = L.bsq_rope_inv_freq(D, 500000.0)[0]
    kc, vc = np.zeros((many, H, page, D), np.uint8), np.zeros((many, H, D, page), np.uint8)
    ks, vs = np.zeros((many, H), np.float32), np.zeros((many, H), np.float32)
    dev = [gpu(a) for a in (np.array([n], np.int32), table, kc, vc, ks, vs)]
    kr, _ = rotate(f64(k), range(n - T, n), f64(w), interleaved, 1.25)
    lens, cu = np.array([n], np.int64), starts([T])
    serve.append(kr, f64(v), cu, lens, table, kc, vc, ks, vs)
    L.bsq_kv_append(k.cuda(), v.cuda(), gpu(cu), *dev, w.cuda(), L.BSQ_ROPE_INTERLEAVED if interleaved else L.BSQ_ROPE_HALF, 1.25)
    assert np.array_equal(f64(dev[4]), ks) and np.array_equal(f64(dev[5]), vs)
    assert np.array_equal(dev[3].cpu().numpy(), vc)
    got = dev[2].cpu().numpy()
    assert np.array_equal(got, kc), "%d of %d codes differ" % ((got != kc).sum(), T * H * D)
