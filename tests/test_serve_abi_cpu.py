"""CPU checks of the token-serving C ABI (include/bsq_serve.h): symbols, the host function against the oracle, and
every refusal, before any HIP call. Pointers are fake and never dereferenced; calls with valid arguments are made
only where there is no GPU, where they report BSQ_ERR_DEVICE."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from block_scaled_precision_row_amd import _lib
from oracle import serve

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = _lib.lib
OK, NULL, SHAPE, ALIGN, WS, DEV, HIP, ARG = range(8)
A, ODD = 1 << 20, (1 << 20) + 2
BF16, FP16, FP32 = _lib.BSQ_BF16, _lib.BSQ_FP16, _lib.BSQ_FP32


def test_every_declared_symbol_is_exported_and_bound():
    with open(os.path.join(ROOT, "include", "bsq_serve.h")) as f:
        syms = sorted(set(re.findall(r"^(?:bsq_status|size_t) (bsq_[a-z0-9_]+)\(", f.read(), re.M)))
    assert syms == ["bsq_attention_kv8", "bsq_attention_kv8_workspace_bytes", "bsq_gemm_int4g", "bsq_kv_append",
                    "bsq_rope", "bsq_rope_inv_freq"]
    for s in syms:
        assert hasattr(ctypes.CDLL(_lib.LIB_PATH), s) and s in _lib.SIGNATURES


@pytest.mark.parametrize("kind,name,kw", [
    (_lib.BSQ_ROPE_PLAIN, "plain", {}), (_lib.BSQ_ROPE_LINEAR, "linear", {"factor": 4.0}),
    (_lib.BSQ_ROPE_NTK, "ntk", {"factor": 8.0}),
    (_lib.BSQ_ROPE_YARN, "yarn", {"factor": 16.0, "trained": 4096}),
    (_lib.BSQ_ROPE_YARN, "yarn", {"factor": 2.5, "trained": 8192, "fast": 48.0, "slow": 0.5})])
@pytest.mark.parametrize("rot", [4, 64, 128])
def test_frequencies(kind, name, kw, rot):
    ref, factor = serve.rope_frequencies(rot, 10000.0, name, kw.get("factor", 1.0), kw.get("trained", 0),
                                         kw.get("fast", 32.0), kw.get("slow", 1.0))
    got, f = _lib.bsq_rope_inv_freq(rot, 10000.0, kind, kw.get("factor", 1.0), kw.get("trained", 0),
                                    kw.get("fast", 32.0), kw.get("slow", 1.0))
    # one rounding to fp32, and a few fp64 ones before it
    assert np.all(np.abs(got.double().numpy() - ref) <= (2.0 ** -24 + 2.0 ** -48) * ref)
    assert abs(f - factor) <= 2.0 ** -24 * factor


def test_frequencies_refusals():
    out, f = torch.empty(64), ctypes.c_float()
    g = lambda r=64, b=1e4, s=0, k=1.0, t=0, bf=32.0, bs=1.0, o=out.data_ptr(), p=ctypes.addressof(f): (  # noqa: E731
        L.bsq_rope_inv_freq(r, b, s, k, t, bf, bs, o, p))
    assert g() == OK and g(o=None) == NULL and g(p=None) == NULL
    assert g(r=63) == SHAPE and g(r=0) == SHAPE and g(r=1026) == SHAPE and g(r=2, s=2, k=2.0) == SHAPE
    assert g(s=4) == ARG and g(s=-1) == ARG and g(b=1.0) == ARG and g(b=float("inf")) == ARG and g(b=float("nan")) == ARG
    assert g(k=2.0) == ARG and g(s=1, k=0.5) == ARG and g(s=1, k=float("nan")) == ARG
    yarn = dict(s=3, k=4.0)
    assert g(t=4096, **yarn) == OK and g(t=0, **yarn) == ARG
    assert g(t=4096, bf=1.0, **yarn) == ARG and g(t=4096, bs=-1.0, **yarn) == ARG
    assert g(t=4096, bf=float("inf"), **yarn) == ARG
    with pytest.raises(_lib.BsqError):
        _lib.bsq_rope_inv_freq(3, 1e4)


def rope(dt=BF16, x=A, xt=512, xh=64, pos=A, freq=A, rot=64, layout=1, f=1.0, flags=0, y=A + (1 << 19), yt=512, yh=64,
         T=4, H=8, D=64):
    return L.bsq_rope(dt, x, xt, xh, pos, freq, rot, layout, f, flags, y, yt, yh, T, H, D, None)


def test_rope_refusals():
    assert rope(dt=0) == ARG and rope(dt=4) == ARG and rope(layout=0) == ARG and rope(layout=3) == ARG
    assert rope(flags=2) == ARG and rope(f=float("inf")) == ARG and rope(f=float("nan")) == ARG
    for bad in ({"rot": 3}, {"rot": 0}, {"rot": -2}, {"rot": 66}, {"D": 0, "rot": 2}, {"D": 1026}, {"T": -1}, {"H": -1},
                {"H": 65536}, {"T": 1 << 31}, {"xt": -512}, {"xh": 1 << 40}, {"yt": -1}):
        assert rope(**bad) == SHAPE, bad
    assert rope(yh=32) == SHAPE and rope(yt=256) == SHAPE and rope(yt=0) == SHAPE   # outputs that overlap
    assert rope(y=A, yt=1024) == SHAPE                                            # in place with other strides
    for p in ("x", "y", "pos", "freq"):
        assert rope(**{p: None}) == NULL
    assert rope(x=A + 1) == ALIGN and rope(dt=FP32, x=ODD) == ALIGN and rope(pos=A + 4) == ALIGN and rope(freq=ODD) == ALIGN
    assert rope(T=0, x=None, y=None) == OK and rope(H=0, x=None, y=None, pos=None) == OK
    if not torch.cuda.is_available():
        assert rope() == DEV and rope(xt=0, xh=0) == DEV and rope(y=A) == DEV       # broadcast input, in place
        assert rope(yt=64, yh=256) == DEV and rope(x=ODD) == DEV                    # heads outermost, any alignment


def cache(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, block_table=A, seq_lens=A, num_pages=10, kv_heads=2, page_size=16,
             head_dim=64, batch=3, max_pages=4, table_stride=4)
    f.update(kw)
    return _lib.Kv8Cache(*[f[n] for n, _ in _lib.Kv8Cache._fields_])


BAD_CACHES = [{"head_dim": 96}, {"head_dim": 0}, {"page_size": 8}, {"page_size": 48}, {"page_size": 512}, {"kv_heads": 0},
              {"kv_heads": 1025}, {"num_pages": 0}, {"num_pages": 1 << 31}, {"batch": -1}, {"batch": 65537},
              {"max_pages": 0}, {"max_pages": 1 << 27, "table_stride": 1 << 27}, {"table_stride": 3}]


def append(dt=BF16, c=None, cu=A, T=5, k=A, kt=128, kh=64, v=A, vt=128, vh=64, freq=A, rot=64, layout=1, f=1.0, q=A,
           qt=256, qh=64, hq=4, qo=A + (1 << 19), ot=256, oh=64, **kw):
    return L.bsq_kv_append(dt, cache(**kw) if c is None else c, cu, T, k, kt, kh, v, vt, vh, freq, rot, layout, f, q, qt, qh,
                           hq, qo, ot, oh, None)


def test_append_refusals():
    assert append(dt=FP32) == ARG and append(layout=7) == ARG and append(f=float("nan")) == ARG
    assert L.bsq_kv_append(BF16, None, A, 5, A, 128, 64, A, 128, 64, None, 0, 1, 1.0, None, 0, 0, 0, None, 0, 0, None) == NULL
    for bad in BAD_CACHES:
        assert append(**bad) == SHAPE, bad
    for bad in ({"T": -1}, {"T": 1 << 31}, {"rot": 8}, {"rot": 80}, {"rot": -16}, {"kt": 4}, {"kh": 12}, {"vt": -8},
                {"vh": 1 << 40}, {"hq": 0}, {"hq": 65536}, {"qt": 12}, {"oh": 32}, {"ot": 128}, {"T": 1 << 24}):
        assert append(**bad) == SHAPE, bad
    assert append(qo=A, ot=512) == SHAPE                                            # in place with other strides
    for p in ("k", "v", "k_scale", "v_scale", "block_table", "seq_lens"):
        assert append(**{p: None}) == NULL and append(**{p: A + 2}) == ALIGN
    assert append(cu=None) == NULL and append(freq=None) == NULL and append(q=None) == NULL and append(qo=None) == NULL
    assert append(q=None, qo=None) == NULL                                        # heads without queries
    assert append(k=A + 4) == ALIGN and append(q=A + 8) == ALIGN and append(cu=ODD) == ALIGN and append(freq=ODD) == ALIGN
    assert append(T=0, k=None, cu=None) == OK and append(batch=0, v=None) == OK
    if not torch.cuda.is_available():
        assert append() == DEV and append(q=None, qo=None, hq=0) == DEV and append(rot=0, freq=None) == DEV
        assert append(qo=A) == DEV and append(kt=0, vt=0) == DEV


def attend(dt=BF16, cu=A, T=5, most=2, q=A, qt=256, qh=64, hq=4, scale=0.125, window=0, flags=0, y=A, yt=256, yh=64, lse=A,
           ws=A, n=None, **kw):
    c = cache(**kw)
    if n is None:
        n = L.bsq_attention_kv8_workspace_bytes(c.batch, T, most, hq, c.kv_heads, c.head_dim)
    return L.bsq_attention_kv8(dt, c, cu, T, most, q, qt, qh, hq, scale, window, flags, y, yt, yh, lse, ws, n, None)


def test_attention_refusals():
    assert attend(dt=FP32) == ARG and attend(flags=2) == ARG and attend(scale=float("inf")) == ARG
    assert attend(window=-1) == ARG and attend(window=4, flags=1) == ARG
    assert L.bsq_attention_kv8(BF16, None, A, 5, 2, A, 256, 64, 4, 0.1, 0, 0, A, 256, 64, A, A, 1 << 30, None) == NULL
    for bad in BAD_CACHES:
        assert attend(n=1 << 40, **bad) == SHAPE, bad
    for bad in ({"T": -1}, {"most": -1}, {"most": 0}, {"hq": 3}, {"hq": 0}, {"hq": 1 << 16}, {"qt": 4}, {"qh": -8}, {"yh": 32},
                {"yt": 128}):
        assert attend(n=1 << 40, **bad) == SHAPE, bad
    for p in ("k", "v", "k_scale", "v_scale", "block_table", "seq_lens"):
        assert attend(**{p: None}) == NULL and attend(**{p: A + 2}) == ALIGN
    assert attend(cu=None) == NULL and attend(q=None) == NULL and attend(y=None) == NULL
    assert attend(q=A + 8) == ALIGN and attend(y=A + 8) == ALIGN and attend(lse=ODD) == ALIGN
    need = L.bsq_attention_kv8_workspace_bytes(3, 5, 2, 4, 2, 64)
    assert need > 0 and need % 256 == 0
    assert attend(n=need - 1) == WS and attend(ws=None) == WS and attend(ws=A + 16) == ALIGN
    assert L.bsq_attention_kv8_workspace_bytes(3, 5, 2, 5, 2, 64) == 0               # a shape that the call refuses
    assert attend(T=0, q=None, y=None, most=0) == OK and attend(batch=0, q=None) == OK
    if not torch.cuda.is_available():
        assert attend() == DEV and attend(lse=None) == DEV and attend(flags=1) == DEV and attend(window=1 << 40) == DEV


def int4(dt=BF16, x=A, ldx=256, w=A, s=A, z=A, group=64, y=A, ldy=48, M=2, N=48, K=256):
    return L.bsq_gemm_int4g(dt, x, ldx, w, s, z, group, y, ldy, M, N, K, None)


def test_int4_refusals():
    assert int4(dt=FP32) == ARG and int4(group=16) == ARG and int4(group=256) == ARG and int4(group=0) == ARG
    for bad in ({"K": 0}, {"K": 224}, {"K": 1 << 21, "ldx": 1 << 21}, {"ldx": 248}, {"ldx": 260}, {"ldy": 47}, {"M": -1},
                {"N": -1}, {"M": 1 << 31}):
        assert int4(**bad) == SHAPE, bad
    assert int4(x=None) == NULL and int4(w=None) == NULL and int4(s=None) == NULL and int4(y=None) == NULL
    assert int4(x=A + 8) == ALIGN and int4(w=A + 8) == ALIGN and int4(s=A + 1) == ALIGN and int4(y=A + 2) == ALIGN
    assert int4(M=0, x=None) == OK and int4(N=0, w=None, ldy=0) == OK
    if not torch.cuda.is_available():
        assert int4() == DEV and int4(z=None) == DEV and int4(K=32, group=32, z=A + 1) == DEV


def test_binding_refuses_tensors_that_do_not_match():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        _lib.bsq_rope(x, torch.zeros(2, dtype=torch.int64), torch.ones(32))          # not on the GPU
    with pytest.raises(ValueError):
        _lib.bsq_kv_append(x, x, i, i, i[None], x, x, x, x)
    with pytest.raises(ValueError):
        _lib.bsq_attention_kv8(x, i, i, i[None], x, x, x, x, 1)
    with pytest.raises(ValueError):
        _lib.bsq_gemm_int4g(x[0].float(), x, x)
