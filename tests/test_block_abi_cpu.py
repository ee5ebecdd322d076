"""CPU checks of the C ABI of a transformer block's operators (include/bsq_block.h): symbols, and every refusal, before
any HIP call. Pointers are fake and never dereferenced; calls with valid arguments are made only where there is no GPU,
where they report BSQ_ERR_DEVICE."""
import ctypes
import os
import re

import torch

from block_scaled_precision_row_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
L = _lib.lib
OK, NULL, SHAPE, ALIGN, WS, DEV, HIP, ARG = range(8)
A, B, ODD = 1 << 20, 1 << 21, (1 << 20) + 2
BF16, FP16, FP32 = _lib.BSQ_BF16, _lib.BSQ_FP16, _lib.BSQ_FP32
NO_GPU = not torch.cuda.is_available()


def test_every_declared_symbol_is_exported_and_bound():
    with open(os.path.join(ROOT, "include", "bsq_block.h")) as f:
        syms = sorted(set(re.findall(r"^(?:bsq_status|size_t) (bsq_[a-z0-9_]+)\(", f.read(), re.M)))
    assert syms == ["bsq_block_norm", "bsq_block_norm_backward", "bsq_block_norm_workspace_bytes",
                    "bsq_gemm_fp8r_q_epilogue", "bsq_gemm_nvfp4_q_epilogue", "bsq_rope_axes"]
    for s in syms:
        assert hasattr(ctypes.CDLL(_lib.LIB_PATH), s) and s in _lib.SIGNATURES


def test_structs_are_laid_out_as_the_header_has_them(tmp_path):
    import shutil
    import subprocess
    if not shutil.which("g++"):
        return
    src = tmp_path / "s.cpp"
    src.write_text('#include <cstdio>\n#include <cstddef>\ntypedef void* hipStream_t;\n#include "bsq_block.h"\nint main() {\n'
                   + "".join('  std::printf("%%zu ", offsetof(bsq_block, %s));\n' % n for n, _ in _lib.Block._fields_)
                   + '  std::printf("%zu\\n", sizeof(bsq_block));\n'
                   + "".join('  std::printf("%%zu ", offsetof(bsq_epilogue, %s));\n' % n for n, _ in _lib.Epilogue._fields_)
                   + '  std::printf("%zu\\n", sizeof(bsq_epilogue));\n}\n')
    hip = tmp_path / "hip"
    hip.mkdir()
    (hip / "hip_runtime_api.h").write_text("")
    subprocess.run(["g++", "-I" + str(tmp_path), "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")],
                   check=True)
    lines = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.splitlines()
    for line, s in zip(lines, (_lib.Block, _lib.Epilogue)):
        assert [int(v) for v in line.split()] == [getattr(s, n).offset for n, _ in s._fields_] + [ctypes.sizeof(s)]


def rope(dt=BF16, x=A, xt=512, xh=64, pos=A, pt=3, pa=1, sections=(8, 12, 12), axes=None, order=1, freq=A, layout=1, f=1.0,
         flags=0, y=A + (1 << 19), yt=512, yh=64, T=4, H=8, D=64):
    s = None if sections is None else (ctypes.c_int64 * len(sections))(*sections)
    return L.bsq_rope_axes(dt, x, xt, xh, pos, pt, pa, s, len(sections) if axes is None else axes, order, freq, layout, f,
                           flags, y, yt, yh, T, H, D, None)


def test_rope_axes_refusals():
    assert rope(dt=0) == ARG and rope(layout=3) == ARG and rope(flags=2) == ARG and rope(f=float("nan")) == ARG
    assert rope(order=0) == ARG and rope(order=3) == ARG
    assert rope(sections=None, axes=3) == NULL
    for bad in ({"axes": 0}, {"axes": 5}, {"sections": (8, -1, 12)}, {"sections": (0, 0)}, {"sections": (33,)},
                {"sections": (513,), "D": 1024, "xh": 1024, "yh": 1024}, {"pt": -1}, {"pa": -1}, {"pt": 1 << 40},
                {"sections": (1, 12, 12), "order": 2}, {"sections": (0, 8), "order": 2}, {"D": 0}, {"T": -1},
                {"H": 65536}, {"xt": -512}, {"yh": 32}, {"yt": 0}, {"y": A, "yt": 1024}):
        assert rope(**bad) == SHAPE, bad
    for p in ("x", "y", "pos", "freq"):
        assert rope(**{p: None}) == NULL
    assert rope(x=A + 1) == ALIGN and rope(dt=FP32, x=ODD) == ALIGN and rope(pos=A + 4) == ALIGN and rope(freq=ODD) == ALIGN
    assert rope(T=0, x=None, y=None) == OK and rope(H=0, x=None, pos=None) == OK
    if NO_GPU:
        assert rope() == DEV and rope(sections=(12, 10, 10), order=2) == DEV and rope(sections=(32,)) == DEV
        assert rope(pt=0, pa=0) == DEV and rope(sections=(0, 16, 0, 16)) == DEV and rope(y=A, xt=512) == DEV


def block(**kw):
    f = dict(dtype=BF16, norm=1, post=0, eps=1e-6, post_eps=1e-6, rows=4, dim=64, groups=1)
    f.update(kw)
    b = _lib.Block()
    for k, v in f.items():
        setattr(b, k, v)
    return b


def norm(x=A, xs=64, h=None, hs=64, xo=None, os_=64, fmt=0, yg=None, y=B, ys=64, ysc=None, **kw):
    return L.bsq_block_norm(block(**kw), x, xs, h, hs, xo, os_, fmt, yg, y, ys, ysc, None)


BRANCH = dict(h=A, xo=B + 4096)
BAD_BLOCKS = [({"dtype": 0}, ARG), ({"dtype": 4}, ARG), ({"norm": 3}, ARG), ({"post": -1}, ARG), ({"eps": -1.0}, ARG),
              ({"eps": float("nan")}, ARG), ({"post_eps": float("inf")}, ARG), ({"post_weight": A}, ARG),
              ({"rows": -1}, SHAPE), ({"rows": 1 << 31}, SHAPE), ({"dim": 0}, SHAPE), ({"dim": 60}, SHAPE),
              ({"dim": 16392}, SHAPE), ({"groups": 0}, SHAPE), ({"groups": 3}, SHAPE), ({"groups": 1 << 25}, SHAPE),
              ({"scale": A, "scale_stride": 12}, SHAPE), ({"shift": A, "shift_stride": -8}, SHAPE),
              ({"groups": 2, "scale": A, "scale_stride": 32}, SHAPE), ({"groups": 2, "shift": A, "shift_stride": 0}, SHAPE),
              ({"weight": ODD}, ALIGN), ({"bias": A + 8}, ALIGN), ({"scale": ODD, "scale_stride": 64}, ALIGN),
              ({"group_starts": ODD}, ALIGN)]


def test_block_norm_refusals():
    assert L.bsq_block_norm(None, A, 64, None, 0, None, 0, 0, None, B, 64, None, None) == NULL
    for bad, status in BAD_BLOCKS:
        assert norm(**bad) == status, bad
    assert norm(fmt=3) == ARG and norm(norm=0) == ARG and norm(norm=0, y=None, fmt=1, **BRANCH) == ARG
    assert norm(norm=0, y=None, weight=A, **BRANCH) == ARG and norm(norm=0, y=None, shift=A, shift_stride=64, **BRANCH) == ARG
    assert norm(gate=A, gate_stride=64) == ARG and norm(xo=B) == ARG and norm(post=2) == ARG   # nothing to gate, add, norm
    assert norm(ysc=A) == ARG and norm(yg=A) == ARG and norm(fmt=1, ysc=A, yg=A) == ARG
    assert norm(fmt=1, ysc=A, dim=72, xs=72) == SHAPE                                         # not a linear's K
    for bad in ({"xs": 32}, {"xs": 68}, {"xs": 1 << 40}, {"xs": -64}, {"ys": 0}, {"ys": 56}, {"h": A, "hs": 8},
                {"h": A, "xo": B, "os_": 0}, {"h": A, "xo": A, "os_": 128}, {"rows": 1 << 25, "dim": 64},
                {"rows": 1 << 23, "dim": 2048, "xs": 2048, "ys": 2048}):
        assert norm(**bad) == SHAPE, bad
    assert norm(x=None) == NULL and norm(y=None) == NULL and norm(fmt=1) == NULL and norm(fmt=2, ysc=A) == NULL
    assert norm(norm=0, y=None, h=A) == NULL                                                  # neither y nor x_out
    assert norm(x=ODD) == ALIGN and norm(y=ODD) == ALIGN and norm(h=A + 8) == ALIGN and norm(fmt=1, ysc=ODD) == ALIGN
    assert norm(fmt=2, ysc=A, yg=ODD) == ALIGN
    assert norm(rows=0, x=None, y=None) == OK
    if NO_GPU:
        assert norm() == DEV and norm(norm=0, y=None, post=1, **BRANCH) == DEV and norm(xs=0) == DEV
        assert norm(fmt=1, ysc=A) == DEV and norm(fmt=2, ysc=A, yg=A) == DEV and norm(h=A, xo=A) == DEV
        assert norm(rows=1, xs=0, ys=0) == DEV and norm(groups=2, scale=A, scale_stride=384) == DEV
        assert norm(rows=5, groups=3, group_starts=A, scale=A, scale_stride=64) == DEV


def back(dy=A, dys=64, do=None, dos=64, xo=A, xos=64, h=None, hs=64, dx=B, dxs=64, dh=None, dhs=64, dsc=None, dsh=None,
         dg=None, dw=None, db=None, dpw=None, ws=A, n=1 << 40, **kw):
    return L.bsq_block_norm_backward(block(**kw), dy, dys, do, dos, xo, xos, h, hs, dx, dxs, dh, dhs, dsc, dsh, dg, dw, db,
                                     dpw, ws, n, None)


def test_block_norm_backward_refusals():
    assert L.bsq_block_norm_backward(None, A, 64, None, 0, A, 64, None, 0, B, 64, None, 0, *[None] * 6, None, 0, None) == NULL
    for bad, status in BAD_BLOCKS:
        assert back(**bad) == status, bad
    for g in ("dsc", "dsh", "dg", "dw", "db", "dpw"):
        assert back(**{g: A}) == ARG                                                          # no such vector
    assert back(norm=0, do=A) == ARG                                                          # dy without a norm
    for bad in ({"dys": 4}, {"xos": 32}, {"do": A, "dos": -8}, {"h": A, "hs": 60}, {"dxs": 0}, {"dh": B, "dhs": 32},
                {"dx": A, "dxs": 128}, {"h": B, "dh": B, "dhs": 128}):
        assert back(**bad) == SHAPE, bad
    assert back(dy=None) == NULL and back(xo=None) == NULL and back(norm=0, dy=None, xo=None) == NULL
    assert back(gate=A, gate_stride=64, dg=A) == NULL and back(post=2, dh=B) == NULL          # no branch
    assert back(post=2, post_weight=A, dpw=A) == NULL
    assert back(dy=ODD) == ALIGN and back(xo=ODD) == ALIGN and back(dx=ODD) == ALIGN and back(do=ODD) == ALIGN
    assert back(weight=A, dw=ODD) == ALIGN
    need = _lib.bsq_block_norm_workspace_bytes(4, 64, 1)
    assert need > 0 and back(weight=A, dw=A, n=need - 1) == WS and back(weight=A, dw=A, ws=None) == WS
    assert back(weight=A, dw=A, ws=A + 16) == ALIGN
    assert back(rows=0, dy=None, xo=None, dx=None) == OK and back(dx=None) == OK
    assert _lib.bsq_block_norm_workspace_bytes(0, 64, 1) == 0 and _lib.bsq_block_norm_workspace_bytes(4, 60, 1) == 0
    assert _lib.bsq_block_norm_workspace_bytes(4, 64, 0) == 0
    if NO_GPU:
        assert back() == DEV and back(ws=None, n=0) == DEV and back(weight=A, dw=A, n=need) == DEV
        assert back(norm=0, dy=None, do=A, xo=None, gate=A, gate_stride=64, h=A, dg=A, dh=B) == DEV
        assert back(dx=A) == DEV and back(dys=0, xos=0) == DEV
        assert back(rows=0, dy=None, xo=None, dx=None, weight=A, dw=A, ws=None) == DEV        # zeros are written


def epi(**kw):
    e = _lib.Epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def fp8r(e, y=B, ldy=64, M=4, N=64, K=64, xq=A, xs=A, w=A, ws=A):
    return L.bsq_gemm_fp8r_q_epilogue(xq, xs, w, ws, e, y, ldy, M, N, K, None)


def nvfp4(e, y=B, ldy=64, M=4, N=64, K=64, xq=A, xs=A, g=A, w=A, ws=A, g2=A):
    return L.bsq_gemm_nvfp4_q_epilogue(xq, xs, g, w, ws, g2, e, y, ldy, M, N, K, None)


def test_epilogue_refusals():
    for f in (fp8r, nvfp4):
        assert f(None) == NULL and f(epi(act=-1)) == ARG and f(epi(act=4)) == ARG
        assert f(epi(), K=48) == SHAPE and f(epi(), ldy=63) == SHAPE and f(epi(), M=-1) == SHAPE
        for p in ("xq", "xs", "w", "ws", "y"):
            assert f(epi(), **{p: None}) == NULL
        assert f(epi(), y=ODD) == ALIGN and f(epi(bias=A + 1)) == ALIGN and f(epi(residual=ODD, residual_stride=64)) == ALIGN
        assert f(epi(gate=A + 1, groups=1)) == ALIGN and f(epi(gate=A, groups=2, gate_stride=64, group_starts=ODD)) == ALIGN
        for bad in (epi(gate=A), epi(gate=A, groups=3, gate_stride=64), epi(gate=A, groups=2, gate_stride=63),
                    epi(gate=A, groups=1 << 25, gate_stride=64, group_starts=A), epi(gate=A, groups=1, gate_stride=-1),
                    epi(residual=A, residual_stride=63), epi(residual=B, residual_stride=128)):
            assert f(bad) == SHAPE
        assert f(None, M=0, y=None) == OK
        if NO_GPU:
            assert f(epi()) == DEV and f(epi(act=3, bias=ODD, residual=B, residual_stride=64)) == DEV
            assert f(epi(gate=ODD, groups=2, gate_stride=384)) == DEV
            assert f(epi(gate=A, groups=3, gate_stride=64, group_starts=A)) == DEV
    assert nvfp4(epi(), g=None) == NULL and nvfp4(epi(), g2=None) == NULL


def test_binding_refusals():
    x = torch.zeros(4, 64)
    for f in (lambda: _lib.bsq_block_norm(x), lambda: _lib.bsq_block_norm_backward(x, None, x),
              lambda: _lib.bsq_rope_axes(x[:, None], torch.zeros(4, 1, dtype=torch.int64), torch.zeros(4), [4])):
        try:
            f()
        except ValueError:
            continue
        raise AssertionError("tensors that are not on the GPU")
