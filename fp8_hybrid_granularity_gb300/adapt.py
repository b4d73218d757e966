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
import functools
from dataclasses import dataclass
from typing import Optional

import torch

from . import E4M3, GRAN_1x128, GRAN_ROW, OUT_BF16, OUT_FP32, QTensor, _round4
from . import lib as _lib
from . import lowbit
from .lowbit import _check, _new, _round16, _streamed

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
_BF16, _F32, _EITHER = {torch.bfloat16: OUT_BF16}, {torch.float32: OUT_FP32}, _KIND


def _kind(dtype, what) -> int:
    kind = _KIND.get(dtype)
    if kind is None:
        raise ValueError(f"{what} must be bfloat16 or float32")
    return kind


def _matrix(x, what, kinds, device, shape=None):
    """Shape, row stride and kind of a matrix of one of the types (and of a shape)."""
    kind, size = kinds.get(x.dtype), x.shape
    if kind is not None and len(size) == 2 and x.get_device() == device and (shape is None or size == shape):
        ld, unit = x.stride()
        if unit == 1 or size[1] <= 1:
            return size, ld if size[0] > 1 else _round16(size[1]), kind
    names = " or ".join(str(d).replace("torch.", "") for d in kinds)
    size = "2-D" if shape is None else f"[{shape[0]}, {shape[1]}]"
    raise ValueError(f"{what} must be a {size} {names} tensor on the current CUDA device with unit column stride")


def _param(p, what, cols, device):
    """Address and kind of the norm's weight or bias."""
    kind = _KIND.get(p.dtype)
    if kind is None or p.shape != (cols,) or p.get_device() != device or not p.is_contiguous():
        raise ValueError(f"{what} must be a contiguous bfloat16 or float32 tensor [{cols}] on the current CUDA device")
    return p.data_ptr(), kind


def _params(weight, bias, cols, device):
    """Addresses of weight and bias and their kind."""
    if weight is None:
        return (None, None, OUT_FP32) if bias is None else (None, *_param(bias, "bias", cols, device))
    w, kind = _param(weight, "weight", cols, device)
    if bias is None:
        return w, None, kind
    b, kind_b = _param(bias, "bias", cols, device)
    if kind_b != kind:
        raise ValueError("weight and bias must have the same type")
    return w, b, kind


def _address(t):
    return None if t is None else t.data_ptr()


def _result(out, shape, dtype, device):
    """The caller's output, checked, or a new one; its row stride and kind."""
    if out is None:
        return _new(tuple(shape), (shape[1], 1), dtype), shape[1], _kind(dtype, "out")
    _, ld, kind = _matrix(out, "out", _EITHER, device, shape)
    return out, ld, kind


@functools.lru_cache(maxsize=4096)
def _bytes(name, *sizes) -> int:
    """A workspace size of the library, a function of sizes alone."""
    return getattr(_fns(), name)(*sizes)


@_streamed
def layernorm(x, weight=None, bias=None, eps: float = 1e-5, out=None, out_dtype=None):
    """y = (x - mean) rstd weight + bias of every row of x [rows, cols], BF16 or
    FP32, in out_dtype (x's), and stats [rows, 2], mean and rstd in FP32, for
    layernorm_bwd."""
    device = lowbit._cuda_device()
    shape, ld, kind = _matrix(x, "x", _EITHER, device)
    rows, cols = shape
    w, b, kind_p = _params(weight, bias, cols, device)
    y, ld_y, kind_y = _result(out, shape, out_dtype or x.dtype, device)
    stats = _new((rows, 2), (2, 1), torch.float32)
    _check((_bound or _fns()).fp8hg_layernorm(x.data_ptr(), kind, rows, cols, ld, w, b, kind_p, eps, y.data_ptr(), kind_y, ld_y, None,
                                              stats.data_ptr(), lowbit._raw_stream(device)), "layernorm")
    return y, stats


@_streamed
def fp8_layernorm(x, weight=None, bias=None, eps: float = 1e-5, group: int = 0, fmt: int = E4M3, with_y: bool = False):
    """The layer norm of x as the A operand of an FP8 product, quantized from FP32
    like fp8_quant_token: one UE8M0 scale per token (group=0) or per 128 columns
    (128; any number of columns, the last group may be shorter).  with_y=True also
    gives y in BF16, from the same read: QTensor, y or None, stats.  Any number of
    rows and columns is quantized; fp8_gemm_scaled takes an operand whose rows and
    columns are multiples of 128, so x of a batch that feeds it is padded to them."""
    device = lowbit._cuda_device()
    shape, ld, kind = _matrix(x, "x", _EITHER, device)
    rows, cols = shape
    w, b, kind_p = _params(weight, bias, cols, device)
    ld_q = _round16(cols)
    if group == 128:
        groups = (cols + 127) // 128
        ld_s = _round4(groups)
        q = QTensor(_new((rows, cols), (ld_q, 1), torch.uint8), _new((rows, ld_s), (ld_s, 1), torch.uint8), fmt, GRAN_1x128, groups)
    elif group == 0:
        ld_s = 1
        q = QTensor(_new((rows, cols), (ld_q, 1), torch.uint8), _new((rows, 1), (1, 1), torch.uint8), fmt, GRAN_ROW, 1)
    else:
        raise ValueError("group must be 0 or 128")
    y = _new((rows, cols), (cols, 1), torch.bfloat16) if with_y else None
    stats = _new((rows, 2), (2, 1), torch.float32)
    codes = _Codes(q.codes.data_ptr(), q.scale.data_ptr(), ld_q, max(1, ld_s), group, fmt)
    _check((_bound or _fns()).fp8hg_layernorm(x.data_ptr(), kind, rows, cols, ld, w, b, kind_p, eps, _address(y), OUT_BF16, cols,
                                              ctypes.byref(codes), stats.data_ptr(), lowbit._raw_stream(device)), "fp8_layernorm")
    return q, y, stats


@_streamed
def layernorm_bwd(dy, x, weight, stats, add=None, out=None, params: bool = True):
    """dx (x's type), dweight and dbias (FP32) from dy, x and the forward pass's
    stats.  add: another branch's gradient of x, added to dx.  out may be add, x
    or dy.
    params=False: dx alone, (dx, None, None)."""
    device = lowbit._cuda_device()
    shape, ld_x, kind = _matrix(x, "x", _EITHER, device)
    rows, cols = shape
    _, ld_dy, kind_dy = _matrix(dy, "dy", _EITHER, device, shape)
    w, _, kind_p = _params(weight, None, cols, device)
    if stats.dtype != torch.float32 or stats.shape != (rows, 2) or stats.get_device() != device or not stats.is_contiguous():
        raise ValueError(f"stats must be a contiguous float32 tensor [{rows}, 2] on the current CUDA device")
    same = _BF16 if kind == OUT_BF16 else _F32
    ld_add = 0 if add is None else _matrix(add, "add", same, device, shape)[1]
    if out is None:
        out, ld_dx = _new((rows, cols), (cols, 1), x.dtype), cols
    else:
        ld_dx = _matrix(out, "out", same, device, shape)[1]
    stream, dw, db, ws, n = lowbit._raw_stream(device), None, None, None, 0
    if params:
        dw, db = _new((cols,), (1,), torch.float32), _new((cols,), (1,), torch.float32)
        n = _bytes("fp8hg_layernorm_bwd_workspace", rows, cols)
        if n:
            ws = lowbit._scratch(n, x, stream)        # held until the call returns
    _check((_bound or _fns()).fp8hg_layernorm_bwd(dy.data_ptr(), kind_dy, ld_dy, x.data_ptr(), kind, ld_x, rows, cols, w, kind_p,
                                                  stats.data_ptr(), _address(add), ld_add, out.data_ptr(), ld_dx, _address(dw),
                                                  _address(db), _address(ws), n, stream), "layernorm_bwd")
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

    def operand(self, device=None) -> _Lora:
        a, b, scale, ranks = self.a, self.b, self.scale, self.ranks
        device = lowbit._cuda_device() if device is None else device
        if not (a.dtype == b.dtype == torch.bfloat16 and a.dim() == b.dim() == 3 and a.get_device() == device and b.get_device() == device):
            raise ValueError("A and B must be 3-D bfloat16 tensors on the current CUDA device")
        g, r, k = a.shape
        g_b, n, r_b = b.shape
        if g_b != g or r_b != r:
            raise ValueError("A [adapters, r, k] and B [adapters, n, r] must have the same adapters and rank")
        stride_a, ld_a, unit_a = a.stride()
        stride_b, ld_b, unit_b = b.stride()
        if (unit_a != 1 and k > 1) or (unit_b != 1 and r > 1):
            raise ValueError("A and B must have unit stride along k and r")
        if scale is not None and (scale.dtype != torch.float32 or scale.shape != (g,) or scale.get_device() != device or not scale.is_contiguous()):
            raise ValueError(f"scale must be a contiguous float32 tensor [{g}] on the current CUDA device")
        if ranks is not None and (ranks.dtype != torch.int32 or ranks.shape != (g,) or ranks.get_device() != device or not ranks.is_contiguous()):
            raise ValueError(f"ranks must be a contiguous int32 tensor [{g}] on the current CUDA device")
        # strides of a dimension of one element say nothing
        return _Lora(a.data_ptr(), b.data_ptr(), _address(scale), _address(ranks), g, r, n, k, stride_a if g > 1 else 0,
                     ld_a if r > 1 else _round16(k), stride_b if g > 1 else 0, ld_b if n > 1 else _round16(r))


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
        if self.words.get_device() != lowbit._cuda_device():
            raise ValueError("the plan must be on the current CUDA device")
        return self.words.data_ptr()


@_streamed
def lora_plan(ids, adapters: int) -> LoraPlan:
    """Groups the tokens of a batch by their adapters, ids [tokens] in int32: one
    that is negative, or not below `adapters`, is a token without an adapter.  Made
    once per batch, for every projection of every layer, forward and backward."""
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous() or ids.get_device() != lowbit._cuda_device():
        raise ValueError("ids must be a contiguous int32 tensor [tokens] on the current CUDA device")
    tokens = ids.shape[0]
    if not 1 <= adapters <= MAX_ADAPTERS or tokens > MAX_TOKENS:
        raise ValueError(f"at most {MAX_ADAPTERS} adapters (one at least) and {MAX_TOKENS} tokens")
    f = _fns()
    n = f.fp8hg_lora_plan_bytes(tokens, adapters)
    words = _new((n // 4,), (1,), torch.int32)
    _check(f.fp8hg_lora_plan(ids.data_ptr(), tokens, adapters, words.data_ptr(), n, lowbit._raw_stream(ids.get_device())), "lora_plan")
    return LoraPlan(words, tokens, adapters)


@_streamed
def lora_add(base, x, adapters: LoraAdapters, plan: LoraPlan, out=None, keep: bool = False, out_dtype=None):
    """y[t] = base[t] + scale_g (x[t] A_g^T) B_g^T with the adapter g of token t,
    beside any projection: base [tokens, n] is its product (BF16 or FP32; None:
    zeros, then out_dtype), x [tokens, k] its BF16 input.  out may be base.
    Returns y and, with keep=True, x A^T [tokens, r] in FP32 for lora_add_bwd
    (None otherwise)."""
    device = lowbit._cuda_device()
    w = adapters.operand(device)
    tokens = x.shape[0]
    ld_x = _matrix(x, "x", _BF16, device, (tokens, w.k))[1]
    shape, ld_base, dtype = (tokens, w.n), 0, out_dtype or torch.bfloat16
    if base is not None:
        ld_base = _matrix(base, "base", _EITHER, device, shape)[1]
        dtype = base.dtype
        if out_dtype not in (None, dtype):
            raise ValueError("out_dtype must be base's type")
    out, ld, kind = _result(out, shape, dtype, device)
    if base is not None and out.dtype != dtype:
        raise ValueError("base and out must have the same type")
    p = plan.address(tokens, w.adapters)
    v = _new((tokens, w.r), (w.r, 1), torch.float32) if keep else None
    stream = lowbit._raw_stream(device)
    n = _bytes("fp8hg_lora_workspace", tokens, w.adapters, w.r, w.k)
    ws = lowbit._scratch(n, x, stream) if n else None        # held until the call returns
    _check((_bound or _fns()).fp8hg_lora_add(ctypes.byref(w), p, tokens, x.data_ptr(), ld_x, _address(base), ld_base, out.data_ptr(), ld,
                                             kind, _address(v), w.r, _address(ws), n, stream), "lora_add")
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
    device = lowbit._cuda_device()
    w = adapters.operand(device)
    tokens = dy.shape[0]
    ld_dy = _matrix(dy, "dy", _BF16, device, (tokens, w.n))[1]
    shape, ld_x, ld_v = (tokens, w.k), 0, 0
    if params:
        ld_x = _matrix(x, "x", _BF16, device, shape)[1]
        ld_v = _matrix(v, "v", _F32, device, (tokens, w.r))[1]
    ld_base, dtype = 0, out_dtype or torch.bfloat16
    if base is not None:
        ld_base = _matrix(base, "base", _EITHER, device, shape)[1]
        dtype = base.dtype
        if out_dtype not in (None, dtype):
            raise ValueError("out_dtype must be base's type")
    out, ld, kind = _result(out, shape, dtype, device)
    if base is not None and out.dtype != dtype:
        raise ValueError("base and out must have the same type")
    p = plan.address(tokens, w.adapters)
    da = db = None
    dw_kind = OUT_FP32
    if params:
        dw_kind = _kind(params_dtype, "the gradients of A and B")
        da = _new((w.adapters, w.r, w.k), (w.r * w.k, w.k, 1), params_dtype)
        db = _new((w.adapters, w.n, w.r), (w.n * w.r, w.r, 1), params_dtype)
    stream = lowbit._raw_stream(device)
    n = _bytes("fp8hg_lora_bwd_workspace", tokens, w.adapters, w.r, w.n, w.k)
    ws = lowbit._scratch(n, dy, stream) if n else None        # held until the call returns
    _check((_bound or _fns()).fp8hg_lora_add_bwd(ctypes.byref(w), p, tokens, dy.data_ptr(), ld_dy, _address(x) if params else None, ld_x,
                                                 _address(v) if params else None, ld_v, _address(base), ld_base, out.data_ptr(), ld, kind,
                                                 _address(da), _address(db), dw_kind, _address(ws), n, stream), "lora_add_bwd")
    return out, da, db
