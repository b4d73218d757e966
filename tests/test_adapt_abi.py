"""The entry points of include/fp8hg_adapt.h: the header is strict C99, the
library exports what it declares, and bad arguments are refused before
anything is launched.  No call here reaches the device."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import adapt

OK, INVALID, ALIGN, SHAPE, UNSUP = 0, 1, 2, 3, 4
FAKE = 0x10000   # never dereferenced
BF16, F32 = fp8hg.OUT_BF16, fp8hg.OUT_FP32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8hg_adapt.h")


@pytest.fixture(scope="module")
def lib():
    return adapt._fns()


def test_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M))
    assert names == {"fp8hg_layernorm", "fp8hg_layernorm_bwd_workspace", "fp8hg_layernorm_bwd", "fp8hg_lora_plan_bytes",
                     "fp8hg_lora_plan", "fp8hg_lora_workspace", "fp8hg_lora_add", "fp8hg_lora_bwd_workspace", "fp8hg_lora_add_bwd"}
    for n in names:
        assert hasattr(lib, n), n


def test_header_is_c99_and_structures_match(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "fp8hg_adapt.h"\nint main(void) {'
                   'printf("%d %d", (int)sizeof(fp8hg_norm_codes), (int)sizeof(fp8hg_lora)); return 0; }\n')
    exe = tmp_path / "s"
    r = subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(adapt._Codes), ctypes.sizeof(adapt._Lora)]


def codes(q=FAKE, s=FAKE, ld=128, ld_s=1, group=0, fmt=0):
    return adapt._Codes(q, s, ld, ld_s, group, fmt)


def test_layernorm_refusals(lib):
    def call(x=FAKE, xk=BF16, rows=4, cols=128, ld=128, w=FAKE, b=FAKE, pk=F32, eps=1e-5, y=FAKE, yk=BF16, ldy=128, q=None, stats=FAKE):
        return lib.fp8hg_layernorm(x, xk, rows, cols, ld, w, b, pk, eps, y, yk, ldy, ctypes.byref(q) if q else None, stats, None)
    assert call(x=None) == INVALID and call(x=FAKE + 1) == ALIGN and call(x=FAKE + 2, xk=F32) == ALIGN
    assert call(xk=2) == INVALID and call(pk=-1) == INVALID and call(yk=7) == INVALID
    assert call(rows=-1) == INVALID and call(ld=127) == INVALID and call(ldy=127) == INVALID
    assert call(eps=-1e-5) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(w=FAKE + 2) == ALIGN and call(b=FAKE + 1, pk=BF16) == ALIGN and call(y=FAKE + 1) == ALIGN
    assert call(stats=FAKE + 4) == ALIGN and call(y=None, stats=None) == INVALID
    assert call(rows=2 ** 31) == SHAPE and call(ld=2 ** 31) == SHAPE and call(ldy=2 ** 31) == SHAPE
    assert call(q=codes(q=None)) == INVALID and call(q=codes(s=None)) == INVALID and call(q=codes(q=FAKE + 8)) == ALIGN
    assert call(q=codes(ld=136)) == ALIGN and call(q=codes(ld=112)) == INVALID and call(q=codes(ld_s=0)) == INVALID
    assert call(q=codes(group=64)) == INVALID and call(q=codes(fmt=2)) == INVALID
    assert call(cols=129, ld=129, ldy=129, q=codes(ld=144, group=128)) == INVALID       # two groups
    assert call(q=codes(ld=2 ** 31)) == SHAPE and call(q=codes(ld_s=2 ** 31)) == SHAPE
    assert call(rows=0) == OK and call(cols=0) == OK and call(rows=0, y=None, stats=None) == OK


def test_layernorm_bwd_refusals(lib):
    need = lib.fp8hg_layernorm_bwd_workspace(4, 128)
    assert need > 0 and lib.fp8hg_layernorm_bwd_workspace(0, 128) == 0 and lib.fp8hg_layernorm_bwd_workspace(4, -1) == 0

    def call(dy=FAKE, dk=BF16, ldd=128, x=FAKE, xk=BF16, ldx=128, rows=4, cols=128, w=FAKE, pk=F32, stats=FAKE, add=None, lda=0, dx=FAKE,
             ldo=128, dw=FAKE, db=FAKE, ws=FAKE, wb=need):
        return lib.fp8hg_layernorm_bwd(dy, dk, ldd, x, xk, ldx, rows, cols, w, pk, stats, add, lda, dx, ldo, dw, db, ws, wb, None)
    assert call(dy=None) == INVALID and call(x=None) == INVALID and call(dx=None) == INVALID and call(stats=None) == INVALID
    assert call(dk=2) == INVALID and call(xk=2) == INVALID and call(pk=2) == INVALID
    assert call(ldd=127) == INVALID and call(ldx=127) == INVALID and call(ldo=127) == INVALID and call(add=FAKE, lda=127) == INVALID
    assert call(dy=FAKE + 1) == ALIGN and call(dx=FAKE + 2, xk=F32) == ALIGN and call(add=FAKE + 1, lda=128) == ALIGN
    assert call(stats=FAKE + 4) == ALIGN and call(dw=FAKE + 2) == ALIGN and call(w=FAKE + 2) == ALIGN
    assert call(ws=None) == INVALID and call(wb=need - 1) == INVALID and call(ws=FAKE + 8) == ALIGN
    assert call(rows=2 ** 31) == SHAPE and call(ldd=2 ** 31) == SHAPE
    assert call(cols=0) == OK and call(rows=0, dw=None, db=None) == OK


def test_plan_refusals(lib):
    need = lib.fp8hg_lora_plan_bytes(100, 3)
    assert lib.fp8hg_lora_plan_bytes(-1, 3) == 0 and lib.fp8hg_lora_plan_bytes(100, 0) == 0
    assert lib.fp8hg_lora_plan_bytes(2 ** 24 + 1, 3) == 0 and lib.fp8hg_lora_plan_bytes(100, 4097) == 0
    call = lambda ids=FAKE, t=100, g=3, p=FAKE, n=need: lib.fp8hg_lora_plan(ids, t, g, p, n, None)  # noqa: E731
    assert call(ids=None) == INVALID and call(ids=FAKE + 2) == ALIGN and call(t=-1) == INVALID and call(g=0) == INVALID
    assert call(t=2 ** 24 + 1) == SHAPE and call(g=4097) == SHAPE
    assert call(p=None) == INVALID and call(p=FAKE + 8) == ALIGN and call(n=need - 1) == INVALID


def lora(a=FAKE, b=FAKE, scale=None, ranks=None, g=2, r=16, n=64, k=32, sa=512, la=32, sb=1024, lb=16):
    return adapt._Lora(a, b, scale, ranks, g, r, n, k, sa, la, sb, lb)


BAD_LORA = [(dict(a=None), INVALID), (dict(b=None), INVALID), (dict(a=FAKE + 1), ALIGN), (dict(b=FAKE + 1), ALIGN),
            (dict(scale=FAKE + 2), ALIGN), (dict(ranks=FAKE + 2), ALIGN), (dict(r=0), INVALID), (dict(r=129, lb=129), UNSUP),
            (dict(g=0), INVALID), (dict(g=4097), SHAPE), (dict(n=-1), INVALID), (dict(n=0), SHAPE), (dict(k=0), SHAPE),
            (dict(k=2 ** 31), SHAPE), (dict(n=2 ** 24 + 1), SHAPE), (dict(la=31), INVALID), (dict(lb=15), INVALID), (dict(sa=-1), INVALID), (dict(la=2 ** 31), SHAPE)]


def test_lora_add_refusals(lib):
    need = lib.fp8hg_lora_workspace(10, 2, 16, 32)
    assert need > 0 and lib.fp8hg_lora_workspace(0, 2, 16, 32) == 0 and lib.fp8hg_lora_workspace(10, 2, 129, 32) == 0
    # rows that are no multiple of 8 long have room for a copy
    assert lib.fp8hg_lora_workspace(10, 2, 16, 33) >= need + 10 * 64 * 2

    def call(w=None, p=FAKE, t=10, x=FAKE, ldx=32, base=FAKE, ldb=64, y=FAKE, ldy=64, yk=BF16, v=None, ldv=0, ws=FAKE, wb=need):
        return lib.fp8hg_lora_add(ctypes.byref(w or lora()), p, t, x, ldx, base, ldb, y, ldy, yk, v, ldv, ws, wb, None)
    assert lib.fp8hg_lora_add(None, FAKE, 10, FAKE, 32, None, 0, FAKE, 64, 0, None, 0, FAKE, need, None) == INVALID
    for change, status in BAD_LORA:
        assert call(lora(**change)) == status, change
    assert call(p=None) == INVALID and call(p=FAKE + 8) == ALIGN and call(t=-1) == INVALID and call(t=2 ** 24 + 1) == SHAPE
    assert call(x=None) == INVALID and call(x=FAKE + 1) == ALIGN and call(ldx=31) == INVALID
    assert call(y=None) == INVALID and call(y=FAKE + 2, yk=F32) == ALIGN and call(ldy=63) == INVALID and call(yk=2) == INVALID
    assert call(base=FAKE + 1) == ALIGN and call(ldb=63) == INVALID
    assert call(v=FAKE, ldv=15) == INVALID and call(v=FAKE + 2, ldv=16) == ALIGN
    assert call(ws=None) == INVALID and call(wb=need - 1) == INVALID and call(ws=FAKE + 8) == ALIGN
    assert call(ldx=2 ** 31) == SHAPE and call(t=0) == OK


def test_lora_add_bwd_refusals(lib):
    need = lib.fp8hg_lora_bwd_workspace(10, 2, 16, 64, 32)
    assert need > 0 and lib.fp8hg_lora_bwd_workspace(10, 2, 16, 0, 32) == 0

    def call(w=None, p=FAKE, t=10, dy=FAKE, ldd=64, x=FAKE, ldx=32, v=FAKE, ldv=16, base=None, ldb=0, dx=FAKE, ldo=32, dk=BF16, da=FAKE,
             db=FAKE, gk=F32, ws=FAKE, wb=need):
        return lib.fp8hg_lora_add_bwd(ctypes.byref(w or lora()), p, t, dy, ldd, x, ldx, v, ldv, base, ldb, dx, ldo, dk, da, db, gk, ws,
                                      wb, None)
    for change, status in BAD_LORA:
        assert call(lora(**change)) == status, change
    assert call(p=None) == INVALID and call(t=-1) == INVALID
    assert call(dy=None) == INVALID and call(ldd=63) == INVALID and call(x=None) == INVALID and call(ldx=31) == INVALID
    assert call(v=None) == INVALID and call(ldv=15) == INVALID and call(v=FAKE + 2) == ALIGN
    assert call(base=FAKE, ldb=31) == INVALID and call(ldo=31) == INVALID and call(dx=FAKE + 1) == ALIGN
    assert call(dk=2) == INVALID and call(gk=2) == INVALID and call(da=FAKE + 2) == ALIGN and call(db=FAKE + 1, gk=BF16) == ALIGN
    assert call(ws=None) == INVALID and call(wb=need - 1) == INVALID and call(ws=FAKE + 8) == ALIGN
    assert call(dx=None, da=None, db=None) == OK and call(t=0, da=None, db=None) == OK
