"""The activations to the accuracy that include/bsq_block.h states, finer than the bf16 of an output: with the residual
-bf16(act(v)) the output is the rest, off by the activation's own error (2^-15 of it; gelu below -5: 4e-7; what is below
2^-119 may be 0), one rounding of the sum in fp32 and one of the rest to bf16. All bf16 v from -104 to 104."""
import numpy as np
import pytest
import torch

from oracle import block
from tests.block_util import f64

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from block_scaled_precision_row_amd import _lib as L


def every_bf16(most):
    bits = torch.arange(0, 1 << 15, dtype=torch.int32)
    v = bits.to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v) & (v <= most)]
    return torch.cat([v, -v])


@pytest.mark.parametrize("fmt", ["fp8r", "nvfp4"])
@pytest.mark.parametrize("M", [1, 300])                           # the few-token kernels' epilogue and the tiles'
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_activations_finer_than_bf16(act, M, fmt):
    v = every_bf16(104.0)
    N, K = len(v), 32
    ref = block.activation(f64(v), act)
    near = torch.from_numpy(ref).bfloat16()
    kw = dict(bias=v.cuda(), act={"silu": 1, "gelu_tanh": 2, "gelu": 3}[act], residual=(-near).expand(M, N).contiguous().cuda())
    byte = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    if fmt == "fp8r":
        y = L.bsq_gemm_fp8r_q_epilogue(byte(M, K), one(M), byte(N, K), one(N), **kw)
    else:
        y = L.bsq_gemm_nvfp4_q_epilogue(byte(M, K // 2), byte(M, K // 16), one(1), byte(N, K // 2), byte(N, K // 16), one(1), **kw)
    rest = ref - f64(near)
    tol = (2.0 ** -15 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -8 * np.abs(rest) + 2.0 ** -119
    if act == "gelu":
        tol = tol + np.where(f64(v) < -5, 4e-7, 0.0)
    bad = np.abs(f64(y) - rest[None]) > tol[None]
    assert not bad.any(), (f64(v)[bad.any(0)][:8], f64(y)[0][bad.any(0)][:8], rest[bad.any(0)][:8])
