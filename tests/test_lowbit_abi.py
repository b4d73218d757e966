"""The entry points of include/fp8hg_lowbit.h: the header is strict C99, the
library exports what it declares, and bad arguments are refused before
anything is launched.  No call here reaches the device."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import lowbit

OK, INVALID, ALIGN, SHAPE, UNSUP = 0, 1, 2, 3, 4
FAKE = 0x10000   # never dereferenced
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8hg_lowbit.h")
MX, NV = fp8hg.FP4_MX, fp8hg.FP4_NV
E4M3, E5M2 = fp8hg.E4M3, fp8hg.E5M2


@pytest.fixture(scope="module")
def lib():
    return lowbit._fns()


def test_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert names == {"fp4_scale_bytes", "fp4_tensor_scale_workspace", "fp4_tensor_scale",
                     "fp4_quant", "fp4_dequant", "fp4_gemm_scaled", "fp4_linear_workspace",
                     "fp4_linear", "fp8_swiglu_ckpt", "fp8_swiglu_ckpt_bwd",
                     "fp8_swiglu_ckpt_bwd_q"}
    for n in names:
        assert hasattr(lib, n), n


def test_header_is_c99(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "h.c"
    src.write_text('#include "fp8hg_lowbit.h"\nint main(void) { return (int)sizeof(fp4hg_operand); }\n')
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only",
                        "-I", os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_structures_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "fp8hg_lowbit.h"\nint main(void) {'
                   'printf("%d %d %d", (int)sizeof(fp4hg_operand), (int)sizeof(fp8hg_swiglu_ckpt),'
                   ' (int)sizeof(fp8hg_swiglu_grads)); return 0; }\n')
    exe = tmp_path / "s"
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(c) for c in (lowbit._Fp4Operand, lowbit._Ckpt, lowbit._Grads)]


def test_scale_bytes(lib):
    assert lib.fp4_scale_bytes(1, 1, MX) == 1024 and lib.fp4_scale_bytes(1, 1, NV) == 2048
    assert lib.fp4_scale_bytes(129, 257, MX) == 4096 and lib.fp4_scale_bytes(128, 256, NV) == 2048
    assert lib.fp4_scale_bytes(0, 5, MX) == 0 and lib.fp4_scale_bytes(5, 5, 2) == 0
    assert lib.fp4_linear_workspace(5, 100, MX) == 5 * 64 + 1024 and lib.fp4_linear_workspace(4, 100, MX) == 0
    q = lambda rows, k, kind: fp8hg.alloc_fp4(rows, k, kind, device="cpu")
    for a in ((1, 1, MX), (129, 257, MX), (300, 3584, NV), (128, 256, NV)):
        assert q(*a).scale.numel() == lib.fp4_scale_bytes(*a)


def test_tensor_scale_refusals(lib):
    n = lib.fp4_tensor_scale_workspace()
    call = lambda x=FAKE, rows=4, cols=4, ld=4, s=FAKE, ws=FAKE, wb=n: lib.fp4_tensor_scale(
        x, rows, cols, ld, s, ws, wb, None)
    assert call(x=None) == INVALID and call(x=FAKE + 1) == ALIGN
    assert call(ld=3) == INVALID and call(rows=-1) == INVALID
    assert call(s=None) == INVALID and call(s=FAKE + 2) == ALIGN
    assert call(ws=None) == INVALID and call(ws=FAKE + 8) == ALIGN and call(wb=n - 1) == INVALID


def test_quant_refusals(lib):
    def call(x=FAKE, rows=4, cols=64, ld=64, kind=MX, t=None, q=FAKE, ldq=32, s=FAKE, qt=None,
             ldqt=0, st=None):
        return lib.fp4_quant(x, rows, cols, ld, kind, t, q, ldq, s, qt, ldqt, st, None)
    assert call(x=None) == INVALID and call(x=FAKE + 1) == ALIGN
    assert call(kind=2) == INVALID and call(rows=-1) == INVALID and call(ld=63) == INVALID
    assert call(t=FAKE) == INVALID                                    # MX has no tensor scale
    assert call(kind=NV, t=FAKE + 2) == ALIGN
    assert call(q=None) == INVALID and call(q=None, s=None) == INVALID
    assert call(s=None) == INVALID and call(s=FAKE + 4) == ALIGN
    assert call(q=FAKE + 8) == ALIGN and call(ldq=24) == ALIGN and call(ldq=16) == INVALID
    assert call(qt=FAKE, ldqt=16) == INVALID                          # codes without scales
    assert call(qt=FAKE + 8, ldqt=16, st=FAKE) == ALIGN
    assert call(qt=FAKE, ldqt=0, st=FAKE) == INVALID
    assert call(rows=2 ** 31) == SHAPE
    assert call(rows=65535 * 128 + 1, qt=FAKE, ldqt=2 ** 22 + 16, st=FAKE) == SHAPE
    assert call(rows=0) == OK and call(cols=0) == OK                  # nothing to do


def op(codes=FAKE, scale=FAKE, ts=None, rows=8, k=64, ld=32, kind=MX, reserved=0):
    return lowbit._Fp4Operand(codes, scale, ts, rows, k, ld, kind, reserved)


def test_dequant_refusals(lib):
    call = lambda o=None, out=FAKE, ld=64, kind=0: lib.fp4_dequant(ctypes.byref(o or op()), out, ld, kind, None)
    assert lib.fp4_dequant(None, FAKE, 64, 0, None) == INVALID
    assert call(out=None) == INVALID and call(ld=63) == INVALID and call(kind=2) == INVALID
    assert call(out=FAKE + 1) == ALIGN and call(out=FAKE + 2, kind=1) == ALIGN
    assert call(op(ld=16)) == INVALID and call(op(ld=40)) == ALIGN and call(op(codes=FAKE + 8)) == ALIGN
    assert call(op(kind=3)) == INVALID and call(op(reserved=1)) == INVALID and call(op(ts=FAKE)) == INVALID
    assert call(op(rows=0)) == OK


def test_gemm_refusals(lib):
    def call(a=None, b=None, c=FAKE, ldc=8, out=0, acc=0, opts=None):
        a, b = a or op(), b or op()
        return lib.fp4_gemm_scaled(ctypes.byref(a), ctypes.byref(b), c, ldc, out, acc,
                                   ctypes.byref(opts) if opts else None, None)
    assert call(c=None) == INVALID and call(ldc=7) == INVALID and call(c=FAKE + 1) == ALIGN
    assert call(c=FAKE + 2, out=1) == ALIGN and call(out=2) == INVALID and call(acc=2) == INVALID
    assert call(b=op(kind=NV)) == UNSUP
    assert call(b=op(k=32)) == SHAPE and call(op(k=0), op(k=0)) == SHAPE
    assert call(op(codes=None)) == INVALID and call(b=op(scale=FAKE + 4)) == ALIGN
    assert call(op(rows=2 ** 31)) == SHAPE
    assert call(opts=fp8hg.GemmOpts(0, 2, 0)) == INVALID and call(opts=fp8hg.GemmOpts(0, 0, 1)) == UNSUP
    assert call(op(rows=0)) == OK and call(b=op(rows=0), ldc=0) == OK


def test_linear_refusals(lib):
    need = lib.fp4_linear_workspace(40, 64, MX)

    def call(x=FAKE, rows=40, ld=64, t=None, w=None, y=FAKE, ldy=8, out=0, ws=FAKE, wb=need):
        w = w or op()
        return lib.fp4_linear(x, rows, ld, t, ctypes.byref(w), y, ldy, out, ws, wb, None, None)
    assert call(x=None) == INVALID and call(ld=63) == INVALID and call(t=FAKE) == INVALID
    assert call(y=None) == INVALID and call(ldy=7) == INVALID and call(out=3) == INVALID
    assert call(ws=None) == INVALID and call(wb=need - 1) == INVALID and call(ws=FAKE + 8) == ALIGN
    assert call(w=op(k=0)) == SHAPE and call(w=op(kind=5)) == INVALID
    assert call(rows=0) == OK


def test_swiglu_refusals(lib):
    def call(g=FAKE, u=FAKE, rows=4, cols=128, ld=128, fh=E4M3, h=FAKE, ldh=128, hs=FAKE, lhs=1,
             f=E4M3, ck=(FAKE,) * 4, ldq=128, lds=1):
        return lib.fp8_swiglu_ckpt(g, u, rows, cols, ld, fh, h, ldh, hs, lhs, f, *ck, ldq, lds, None)
    assert call(g=None) == INVALID and call(u=None) == INVALID and call(u=FAKE + 1) == ALIGN
    assert call(ld=127) == INVALID and call(fh=2) == INVALID and call(f=2) == INVALID
    assert call(h=None) == INVALID and call(hs=None) == INVALID and call(h=FAKE + 8) == ALIGN
    assert call(ldh=136) == ALIGN and call(ldh=112) == INVALID and call(lhs=0) == INVALID
    assert call(ck=(FAKE, None, FAKE, FAKE)) == INVALID
    assert call(ck=(FAKE + 4, FAKE, FAKE, FAKE)) == ALIGN and call(ldq=136) == ALIGN
    assert call(ldq=112) == INVALID and call(lds=0) == INVALID
    assert call(rows=0) == OK and call(cols=0) == OK and call(rows=-1) == INVALID


def ck(gq=FAKE, gs=FAKE, uq=FAKE, us=FAKE, rows=128, cols=128, ldq=128, lds=1, fmt=E4M3, reserved=0):
    return lowbit._Ckpt(gq, gs, uq, us, rows, cols, ldq, lds, fmt, reserved)


def test_swiglu_bwd_refusals(lib):
    def call(dh=FAKE, ld=128, c=None, dg=FAKE, du=FAKE, ldd=128):
        c = c or ck()
        return lib.fp8_swiglu_ckpt_bwd(dh, ld, ctypes.byref(c), dg, du, ldd, None)
    assert lib.fp8_swiglu_ckpt_bwd(FAKE, 128, None, FAKE, FAKE, 128, None) == INVALID
    assert call(dh=None) == INVALID and call(ld=127) == INVALID and call(dg=None) == INVALID
    assert call(du=FAKE + 1) == ALIGN and call(ldd=127) == INVALID
    assert call(c=ck(gq=None)) == INVALID and call(c=ck(gq=FAKE + 8)) == ALIGN
    assert call(c=ck(fmt=2)) == INVALID and call(c=ck(lds=0)) == INVALID and call(c=ck(ldq=136)) == ALIGN
    assert call(c=ck(rows=0)) == OK


def test_swiglu_bwd_q_refusals(lib):
    names = [n for n, _ in lowbit._Grads._fields_]
    base = dict({n: FAKE for n in names[:10]}, ld_q=128, ld_s=1, ld_qt=128, ld_st=1, fmt=E5M2,
                fmt_t=E5M2, fmt_h=E4M3, reserved=0)

    def call(dh=FAKE, ld=128, c=None, **change):
        c = c or ck()
        g = lowbit._Grads(**{**base, **change})
        return lib.fp8_swiglu_ckpt_bwd_q(dh, ld, ctypes.byref(c), ctypes.byref(g), None)
    assert call(dh=None) == INVALID and call(dh=FAKE + 2) == ALIGN and call(ld=132) == ALIGN
    assert call(c=ck(rows=130)) == SHAPE and call(c=ck(cols=100)) == SHAPE
    for n in names[:10]:
        assert call(**{n: None}) == INVALID, n
    for n in ("dgate_q", "dup_q", "dgate_qt", "dup_qt", "h_qt"):
        assert call(**{n: FAKE + 8}) == ALIGN, n
    assert call(ld_q=136) == ALIGN and call(ld_qt=136) == ALIGN and call(ld_q=112) == INVALID
    assert call(ld_s=0) == INVALID and call(ld_st=0) == INVALID and call(fmt_h=2) == INVALID
    assert call(reserved=1) == INVALID and call(c=ck(rows=0)) == OK


def test_strides_of_31_bits(lib):
    """Row strides past 2^31 - 1 are refused, not cut."""
    big = 2 ** 31          # a multiple of 16
    n = lib.fp4_tensor_scale_workspace()
    assert lib.fp4_tensor_scale(FAKE, 4, 4, big, FAKE, FAKE, n, None) == SHAPE
    quant = lambda ld=64, ldq=32, ldqt=16: lib.fp4_quant(FAKE, 4, 64, ld, MX, None, FAKE, ldq, FAKE, FAKE, ldqt, FAKE, None)
    assert quant(ld=big) == SHAPE and quant(ldq=big) == SHAPE and quant(ldqt=big) == SHAPE
    dequant = lambda o, ld=64: lib.fp4_dequant(ctypes.byref(o), FAKE, ld, 0, None)
    assert dequant(op(), big) == SHAPE and dequant(op(ld=big)) == SHAPE
    fwd = lambda **k: lib.fp8_swiglu_ckpt(FAKE, FAKE, 4, 128, k.get("ld", 128), E4M3, FAKE, k.get("ldh", 128), FAKE,
                                          k.get("lhs", 1), E4M3, FAKE, FAKE, FAKE, FAKE, k.get("ldq", 128),
                                          k.get("lds", 1), None)
    assert all(fwd(**{k: big}) == SHAPE for k in ("ld", "ldh", "lhs", "ldq", "lds"))
    bwd = lambda ld=128, c=None, ldd=128: lib.fp8_swiglu_ckpt_bwd(FAKE, ld, ctypes.byref(c or ck()), FAKE, FAKE, ldd, None)
    assert bwd(ld=big) == SHAPE and bwd(ldd=big) == SHAPE
    assert bwd(c=ck(ldq=big)) == SHAPE and bwd(c=ck(lds=big)) == SHAPE
    names = [n for n, _ in lowbit._Grads._fields_]
    base = dict({n: FAKE for n in names[:10]}, ld_q=128, ld_s=1, ld_qt=128, ld_st=1, fmt=E5M2,
                fmt_t=E5M2, fmt_h=E4M3, reserved=0)
    for name in ("ld_q", "ld_s", "ld_qt", "ld_st"):
        g = lowbit._Grads(**{**base, name: big})
        assert lib.fp8_swiglu_ckpt_bwd_q(FAKE, 128, ctypes.byref(ck()), ctypes.byref(g), None) == SHAPE, name
