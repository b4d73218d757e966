"""Layer norm and low-rank adapters.

Python binding of ``include/fp8hg_adapt.h`` (the same ``libfp8hg.so``); the
package exports every name here.  As in the rest of the package, arguments are
checked and marshalled and the CUDA kernels do all of the computation.

  layernorm(x, weight, bias, eps)                   -> y, stats
  fp8_layernorm(x, weight, bias, eps, group=0|128)  -> QTensor, y or None, stats
  layernorm_bwd(dy, x, weight, stats, add=None)     -> dx, dweight, dbias
  lora_plan(ids, adapters)                          -> LoraPlan, for all calls on a batch
  lora_add(base, x, adapters, plan, keep=False)     -> y = base + s (x A^T) B^T, x A^T or None
  lora_add_bwd(dy, x, v, adapters, plan, base)      -> dx, dA, dB

Every one takes stream=, a torch stream or a raw handle, as well.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import E4M3, GRAN_1x128, GRAN_ROW, OUT_BF16, OUT_FP32, QTensor
from . import lib as _lib
from . import lowbit
from .lowbit import _check, _groups, _new, _round16, _streamed

MAX_RANK, MAX_ADAPTERS, MAX_TOKENS = 128, 4096, 1 << 24


class _Codes(ctypes.Structure):
    """fp8hg_norm_codes of the C header."""
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("ld_scale", ctypes.c_int64), ("group", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class _Lora(ctypes.Structure):
    """fp8hg_lora of the C header."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("a", "b", "scale", "ranks")] +
                [(n, ctypes.c_int64) for n in ("adapters", "r", "n", "k", "stride_a", "ld_a", "stride_b", "ld_b")])


_bound = None


def _fns():
    """The library with the argument types of this module's functions set."""
    global _bound
    if _bound is None:
        f = _lib()
        P, I64, I, Z, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        f.fp8hg_layernorm.argtypes = [P, I, I64, I64, I64, P, P, I, F, P, I, I64, P, P, P]
        f.fp8hg_layernorm_bwd_workspace.argtypes = [I64, I64]
        f.fp8hg_layernorm_bwd.argtypes = [P, I, I64, P, I, I64, I64, I64, P, I, P, P, I64, P, I64, P, P, P, Z, P]
        f.fp8hg_lora_plan_bytes.argtypes = [I64, I64]
        f.fp8hg_lora_plan.argtypes = [P, I64, I64, P, Z, P]
        f.fp8hg_lora_workspace.argtypes = [I64] * 4
        f.fp8hg_lora_add.argtypes = [P, P, I64, P, I64, P, I64, P, I64, I, P, I64, P, Z, P]
        f.fp8hg_lora_bwd_workspace.argtypes = [I64] * 5
        f.fp8hg_lora_add_bwd.argtypes = [P, P, I64, P, I64, P, I64, P, I64, P, I64, P, I64, I, P, P, I, P, Z, P]
        for n in ("fp8hg_layernorm_bwd_workspace", "fp8hg_lora_plan_bytes", "fp8hg_lora_workspace", "fp8hg_lora_bwd_workspace"):
            getattr(f, n).restype = Z
        _bound = f
    return _bound


_KIND = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32}


def _here(t) -> bool:
    return lowbit._here(t)


def _on(x):
    return lowbit._on(x)


def _kind(dtype, what) -> int:
    kind = _KIND.get(dtype)
    if kind is None:
        raise ValueError(f"{what} must be bfloat16 or float32")
    return kind


def _matrix(x, what, dtypes, shape=None):
    """Rows, columns and row stride of a matrix of one of the types (and of a shape)."""
    if x.dtype in dtypes and x.dim() == 2 and _here(x):
        rows, cols = x.shape
        ld, unit = x.stride()
        if (shape is None or (rows, cols) == shape) and (unit == 1 or cols <= 1):
            return rows, cols, ld if rows > 1 else _round16(cols)
    names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
    size = "2-D" if shape is None else f"[{shape[0]}, {shape[1]}]"
    raise ValueError(f"{what} must be a {size} {names} tensor on the current CUDA device with unit column stride")


_BF16, _F32, _EITHER = (torch.bfloat16,), (torch.float32,), (torch.bfloat16, torch.float32)


def _params(weight, bias, cols):
    """Addresses of weight and bias and their kind."""
    kind = OUT_FP32
    for what, p in (("weight", weight), ("bias", bias)):
        if p is not None:
            if p.dtype not in _KIND or tuple(p.shape) != (cols,) or not _here(p) or (cols > 1 and p.stride(0) != 1):
                raise ValueError(f"{what} must be a contiguous bfloat16 or float32 tensor [{cols}] on the current CUDA device")
            kind = _KIND[p.dtype]
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have the same type")
    return _address(weight), _address(bias), kind


def _address(t):
    return None if t is None else t.data_ptr()


def _result(out, rows, cols, dtype, what="out"):
    """The caller's output, checked, or a new one; its row stride and kind."""
    if out is None:
        return _new((rows, cols), (cols, 1), dtype), cols, _kind(dtype, what)
    _, _, ld = _matrix(out, what, _EITHER, (rows, cols))
    return out, ld, _KIND[out.dtype]


def _scratch(n, x, stream):
    return lowbit._scratch(n, x, stream)


def _norm(x, weight, bias, eps, y, ld_y, y_kind, codes, stats):
    rows, cols, ld = _matrix(x, "x", _EITHER)
    w, b, kind = _params(weight, bias, cols)
    _check(_fns().fp8hg_layernorm(x.data_ptr(), _KIND[x.dtype], rows, cols, ld, w, b, kind, eps, _address(y), y_kind, ld_y,
                                  codes, stats.data_ptr(), _on(x)), "layernorm")


@_streamed
def layernorm(x, weight=None, bias=None, eps: float = 1e-5, out=None, out_dtype=None):
    """y = (x - mean) rstd weight + bias of every row of x [rows, cols], BF16 or
    FP32, in out_dtype (x's), and stats [rows, 2], mean and rstd in FP32, for
    layernorm_bwd."""
    rows, cols, _ = _matrix(x, "x", _EITHER)
    y, ld, kind = _result(out, rows, cols, out_dtype or x.dtype)
    stats = _new((rows, 2), (2, 1), torch.float32)
    _norm(x, weight, bias, eps, y, ld, kind, None, stats)
    return y, stats


@_streamed
def fp8_layernorm(x, weight=None, bias=None, eps: float = 1e-5, group: int = 0, fmt: int = E4M3, with_y: bool = False):
    """The layer norm of x as the A operand of an FP8 product, quantized from FP32
    like fp8_quant_token: one UE8M0 scale per token (group=0) or per 128 columns
    (128; any number of columns, the last group may be shorter).  with_y=True also
    gives y in BF16, from the same read: QTensor, y or None, stats."""
    rows, cols, _ = _matrix(x, "x", _EITHER)
    if group not in (0, 128):
        raise ValueError("group must be 0 or 128")
    if group:
        q = _groups(rows, cols, fmt)
    else:
        q = QTensor(_new((rows, cols), (_round16(cols), 1), torch.uint8), _new((rows, 1), (1, 1), torch.uint8), fmt, GRAN_ROW, 1)
    y = _new((rows, cols), (cols, 1), torch.bfloat16) if with_y else None
    stats = _new((rows, 2), (2, 1), torch.float32)
    codes = _Codes(q.codes.data_ptr(), q.scale.data_ptr(), _round16(cols), max(1, q.scale.stride(0)), group, fmt)
    _norm(x, weight, bias, eps, y, cols, OUT_BF16, ctypes.byref(codes), stats)
    return q, y, stats


@_streamed
def layernorm_bwd(dy, x, weight, stats, add=None, out=None, params: bool = True):
    """dx (x's type), dweight and dbias (FP32) from dy, x and the forward pass's
    stats.  add: another branch's gradient of x, added to dx (may be out).
    params=False: dx alone, (dx, None, None)."""
    rows, cols, ld_x = _matrix(x, "x", _EITHER)
    _, _, ld_dy = _matrix(dy, "dy", _EITHER, (rows, cols))
    w, _, kind = _params(weight, None, cols)
    if stats.dtype != torch.float32 or tuple(stats.shape) != (rows, 2) or not stats.is_contiguous() or not _here(stats):
        raise ValueError(f"stats must be a contiguous float32 tensor [{rows}, 2] on the current CUDA device")
    ld_add = 0 if add is None else _matrix(add, "add", (x.dtype,), (rows, cols))[2]
    if out is None:
        out, ld_dx = _new((rows, cols), (cols, 1), x.dtype), cols
    else:
        ld_dx = _matrix(out, "out", (x.dtype,), (rows, cols))[2]
    dw = _new((cols,), (1,), torch.float32) if params else None
    db = _new((cols,), (1,), torch.float32) if params else None
    f = _fns()
    stream = _on(x)
    n = f.fp8hg_layernorm_bwd_workspace(rows, cols) if params else 0
    ws = _scratch(n, x, stream).data_ptr() if n else None
    _check(f.fp8hg_layernorm_bwd(dy.data_ptr(), _KIND[dy.dtype], ld_dy, x.data_ptr(), _KIND[x.dtype], ld_x, rows, cols, w, kind,
                                 stats.data_ptr(), _address(add), ld_add, out.data_ptr(), ld_dx, _address(dw), _address(db), ws, n,
                                 stream), "layernorm_bwd")
    return out, dw, db


# ------------------------------------------------------------ low-rank adapters
@dataclass
class LoraAdapters:
    """Adapters beside one projection [n, k]: A [adapters, r, k] and B [adapters,
    n, r] in BF16 (unit stride along k and r), scale [adapters] in FP32 (None: 1)
    and ranks [adapters] in int32 (None: r); what lies past an adapter's rank is
    not used."""
    a: torch.Tensor
    b: torch.Tensor
    scale: Optional[torch.Tensor] = None
    ranks: Optional[torch.Tensor] = None

    def operand(self) -> _Lora:
        a, b = self.a, self.b
        if not (a.dtype == b.dtype == torch.bfloat16 and a.dim() == b.dim() == 3 and _here(a) and _here(b)):
            raise ValueError("A and B must be 3-D bfloat16 tensors on the current CUDA device")
        g, r, k = a.shape
        n = b.shape[1]
        if b.shape[0] != g or b.shape[2] != r:
            raise ValueError("A [adapters, r, k] and B [adapters, n, r] must have the same adapters and rank")
        if (k > 1 and a.stride(2) != 1) or (r > 1 and b.stride(2) != 1):
            raise ValueError("A and B must have unit stride along k and r")
        for what, t, dtype in (("scale", self.scale, torch.float32), ("ranks", self.ranks, torch.int32)):
            if t is not None and (t.dtype != dtype or tuple(t.shape) != (g,) or not t.is_contiguous() or not _here(t)):
                raise ValueError(f"{what} must be a contiguous {str(dtype)[6:]} tensor [{g}] on the current CUDA device")
        # strides of a dimension of one element say nothing
        ld_a, ld_b = a.stride(1) if r > 1 else _round16(k), b.stride(1) if n > 1 else _round16(r)
        return _Lora(a.data_ptr(), b.data_ptr(), _address(self.scale), _address(self.ranks), g, r, n, k,
                     a.stride(0) if g > 1 else 0, ld_a, b.stride(0) if g > 1 else 0, ld_b)


@dataclass
class LoraPlan:
    """The tokens of a batch grouped by adapter (lora_plan), on the device; its
    content is the library's."""
    words: torch.Tensor
    tokens: int
    adapters: int

    def address(self, tokens, adapters):
        if (self.tokens, self.adapters) != (tokens, adapters):
            raise ValueError(f"the plan is of {self.tokens} tokens and {self.adapters} adapters, the call of {tokens} and {adapters}")
        if not _here(self.words):
            raise ValueError("the plan must be on the current CUDA device")
        return self.words.data_ptr()


@_streamed
def lora_plan(ids, adapters: int) -> LoraPlan:
    """Groups the tokens of a batch by their adapters, ids [tokens] in int32: one
    that is negative, or not below `adapters`, is a token without an adapter.  Made
    once per batch, for every projection of every layer, forward and backward."""
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous() or not _here(ids):
        raise ValueError("ids must be a contiguous int32 tensor [tokens] on the current CUDA device")
    tokens = ids.shape[0]
    if not 1 <= adapters <= MAX_ADAPTERS or tokens > MAX_TOKENS:
        raise ValueError(f"at most {MAX_ADAPTERS} adapters (one at least) and {MAX_TOKENS} tokens")
    f = _fns()
    n = f.fp8hg_lora_plan_bytes(tokens, adapters)
    words = _new((n // 4,), (1,), torch.int32)
    _check(f.fp8hg_lora_plan(ids.data_ptr(), tokens, adapters, words.data_ptr(), n, _on(ids)), "lora_plan")
    return LoraPlan(words, tokens, adapters)


@_streamed
def lora_add(base, x, adapters: LoraAdapters, plan: LoraPlan, out=None, keep: bool = False, out_dtype=None):
    """y[t] = base[t] + scale_g (x[t] A_g^T) B_g^T with the adapter g of token t,
    beside any projection: base [tokens, n] is its product (BF16 or FP32; None:
    zeros, then out_dtype), x [tokens, k] its BF16 input.  out may be base.
    Returns y and, with keep=True, x A^T [tokens, r] in FP32 for lora_add_bwd
    (None otherwise)."""
    w = adapters.operand()
    tokens, _, ld_x = _matrix(x, "x", _BF16, (x.shape[0], w.k) if x.dim() == 2 else None)
    ld_base, dtype = 0, out_dtype or torch.bfloat16
    if base is not None:
        _, _, ld_base = _matrix(base, "base", _EITHER, (tokens, w.n))
        dtype = base.dtype
        if out_dtype not in (None, dtype):
            raise ValueError("out_dtype must be base's type")
    out, ld, kind = _result(out, tokens, w.n, dtype)
    if base is not None and out.dtype != dtype:
        raise ValueError("base and out must have the same type")
    p = plan.address(tokens, w.adapters)
    v = _new((tokens, w.r), (w.r, 1), torch.float32) if keep else None
    f = _fns()
    stream = _on(x)
    n = f.fp8hg_lora_workspace(tokens, w.adapters, w.r, w.k)
    ws = _scratch(n, x, stream).data_ptr() if n else None
    _check(f.fp8hg_lora_add(ctypes.byref(w), p, tokens, x.data_ptr(), ld_x, _address(base), ld_base, out.data_ptr(), ld, kind,
                            _address(v), w.r, ws, n, stream), "lora_add")
    return out, v


@_streamed
def lora_add_bwd(dy, x, v, adapters: LoraAdapters, plan: LoraPlan, base=None, out=None, out_dtype=None,
                 params: bool = True, params_dtype=torch.float32):
    """dx[t] = base[t] + dv[t] A_g with dv[t] = scale_g dy[t] B_g, dA_g = dv^T x
    [adapters, r, k] and dB_g = scale_g dy^T v [adapters, n, r] over g's tokens.
    dy and x in BF16, v from lora_add(keep=True); base [tokens, k] is the
    projection's own data gradient (None: zeros, then out_dtype); out may be base.
    The gradients of A and B have params_dtype; params=False: dx alone, and x and v
    may be None."""
    w = adapters.operand()
    tokens, _, ld_dy = _matrix(dy, "dy", _BF16, (dy.shape[0], w.n) if dy.dim() == 2 else None)
    ld_x = ld_v = 0
    if params:
        ld_x = _matrix(x, "x", _BF16, (tokens, w.k))[2]
        ld_v = _matrix(v, "v", _F32, (tokens, w.r))[2]
    ld_base, dtype = 0, out_dtype or torch.bfloat16
    if base is not None:
        _, _, ld_base = _matrix(base, "base", _EITHER, (tokens, w.k))
        dtype = base.dtype
        if out_dtype not in (None, dtype):
            raise ValueError("out_dtype must be base's type")
    out, ld, kind = _result(out, tokens, w.k, dtype)
    if base is not None and out.dtype != dtype:
        raise ValueError("base and out must have the same type")
    p = plan.address(tokens, w.adapters)
    da = db = None
    dw_kind = OUT_FP32
    if params:
        dw_kind = _kind(params_dtype, "the gradients of A and B")
        da = _new((w.adapters, w.r, w.k), (w.r * w.k, w.k, 1), params_dtype)
        db = _new((w.adapters, w.n, w.r), (w.n * w.r, w.r, 1), params_dtype)
    f = _fns()
    stream = _on(dy)
    n = f.fp8hg_lora_bwd_workspace(tokens, w.adapters, w.r, w.n, w.k)
    ws = _scratch(n, dy, stream).data_ptr() if n else None
    _check(f.fp8hg_lora_add_bwd(ctypes.byref(w), p, tokens, dy.data_ptr(), ld_dy, _address(x) if params else None, ld_x,
                                _address(v) if params else None, ld_v, _address(base), ld_base, out.data_ptr(), ld, kind,
                                _address(da), _address(db), dw_kind, ws, n, stream), "lora_add_bwd")
    return out, da, db
