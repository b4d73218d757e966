"""4-bit microscaled tensors and SwiGLU with 8-bit activation checkpoints.

Python binding of ``include/fp8hg_lowbit.h`` (the same ``libfp8hg.so``); the
package exports every name here.  As in the rest of the package, arguments are
checked and marshalled and the CUDA kernels do all of the computation.

  fp4_tensor_scale(x)                               -> float32 tensor of one element (FP4_NV)
  fp4_quant(x, kind, tensor_scale, transpose=False) -> Fp4Tensor
  fp4_quant_dual(x, kind, tensor_scale)             -> Fp4Tensor, Fp4Tensor^T (one read)
  fp4_dequant(q, out_dtype=bf16)                    -> values
  fp4_gemm_scaled(a, b, out=None, out_dtype=bf16, accumulate=False)
  fp4_linear(x, w, tensor_scale)                    quantize x and multiply, one call
  fp8_swiglu_ckpt(gate, up, checkpoint=True)        -> QTensor, SwigluCkpt
  fp8_swiglu_ckpt_bwd(dh, ckpt)                     -> [rows, 2 cols] BF16, dgate next to dup
  fp8_swiglu_ckpt_bwd_q(dh, ckpt)                   -> the same as FP8 operands in both
                                                       directions, and h transposed

Every one takes stream=, a torch stream or a raw handle, as well.
"""
from __future__ import annotations

import ctypes
import functools
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import (E4M3, E5M2, GRAN_1x128, OUT_BF16, OUT_FP32, Fp8hgError, GemmOpts, QTensor, _round4,
               _stream)
from . import lib as _lib

FP4_MX, FP4_NV = 0, 1
FP4_BLOCK = {FP4_MX: 32, FP4_NV: 16}


class _Fp4Operand(ctypes.Structure):
    """fp4hg_operand of the C header."""
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("rows", ctypes.c_int64), ("k", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("kind", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _Ckpt(ctypes.Structure):
    """fp8hg_swiglu_ckpt of the C header."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("gate_q", "gate_s", "up_q", "up_s")] +
                [(n, ctypes.c_int64) for n in ("rows", "cols", "ld_q", "ld_s")] +
                [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32)])


class _Grads(ctypes.Structure):
    """fp8hg_swiglu_grads of the C header."""
    _fields_ = ([(n, ctypes.c_void_p) for n in
                 ("dgate_q", "dup_q", "dgate_s", "dup_s", "dgate_qt", "dup_qt", "dgate_st",
                  "dup_st", "h_qt", "h_st")] +
                [(n, ctypes.c_int64) for n in ("ld_q", "ld_s", "ld_qt", "ld_st")] +
                [(n, ctypes.c_int32) for n in ("fmt", "fmt_t", "fmt_h", "reserved")])


_bound = None
_raw_stream = torch._C._cuda_getCurrentRawStream


_cuda_device = torch._C._cuda_getDevice


def _here(t) -> bool:
    """Whether t is on the current device: the one that a call launches on, and
    whose memory it may touch."""
    return t.get_device() == _cuda_device()   # -1 on the CPU


# the allocation (sizes, strides, type) on the current device; torch.empty without
# its argument handling: in a row of small calls an output costs the host 1.4 us
# instead of 4
_new = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)
if _new is None:
    def _new(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _on(x):
    """The stream to launch on, x's device's current one (the plain lookup: a
    call takes about as long as ten microseconds' work)."""
    return _raw_stream(x.get_device())


def _streamed(fn):
    """Adds the keyword `stream` (a torch stream or a raw handle; None: the
    current one): the call runs with it as the current stream, so that what it
    allocates belongs to that stream and no other stream's pending work on
    reused memory can reach it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            # 0 is the default stream; ExternalStream(0) would be a new one
            handle = _stream(stream)
            stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _check(rc: int, what: str):
    if rc != 0:
        raise Fp8hgError(what, rc)


def _fns():
    """The library with the argument types of this module's functions set."""
    global _bound
    if _bound is None:
        f = _lib()
        P, I64, I, Z = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        f.fp4_scale_bytes.argtypes = [I64, I64, I]
        f.fp4_scale_bytes.restype = Z
        f.fp4_tensor_scale_workspace.argtypes = []
        f.fp4_tensor_scale_workspace.restype = Z
        f.fp4_tensor_scale.argtypes = [P, I64, I64, I64, P, P, Z, P]
        f.fp4_quant.argtypes = [P, I64, I64, I64, I, P, P, I64, P, P, I64, P, P]
        f.fp4_dequant.argtypes = [P, P, I64, I, P]
        f.fp4_gemm_scaled.argtypes = [P, P, P, I64, I, I, P, P]
        f.fp4_linear_workspace.argtypes = [I64, I64, I]
        f.fp4_linear_workspace.restype = Z
        f.fp4_linear.argtypes = [P, I64, I64, P, P, P, I64, I, P, Z, P, P]
        f.fp8_swiglu_ckpt.argtypes = [P, P, I64, I64, I64, I, P, I64, P, I64, I, P, P, P, P, I64,
                                      I64, P]
        f.fp8_swiglu_ckpt_bwd.argtypes = [P, I64, P, P, P, I64, P]
        f.fp8_swiglu_ckpt_bwd_q.argtypes = [P, I64, P, P, P]
        _bound = f
    return _bound


def _round16(n: int) -> int:
    """The row stride that a tensor of one row is given: its own says nothing,
    and may be too small, misaligned or unlike another operand's."""
    return (n + 15) // 16 * 16


def _matrix(x, what="x"):
    """Rows, columns and row stride of a BF16 input."""
    if x.dtype == torch.bfloat16 and x.dim() == 2 and _here(x):
        rows, cols = x.shape
        ld, unit = x.stride()
        if unit == 1 or cols <= 1:
            return rows, cols, ld if rows > 1 else _round16(cols)
    raise ValueError(f"{what} must be a 2-D bfloat16 tensor on the current CUDA device with unit column stride")


def _ld(x) -> int:
    """Row stride of an output or of FP8 codes."""
    return x.stride(0) if x.shape[0] > 1 else _round16(x.shape[1])


def _ts(t):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1 or not _here(t):
        raise ValueError("tensor_scale must be a float32 tensor of one element on the current CUDA device")
    return t.data_ptr()


def _out_kind(dtype) -> int:
    if dtype == torch.bfloat16:
        return OUT_BF16
    if dtype == torch.float32:
        return OUT_FP32
    raise ValueError("out must be bfloat16 or float32")


def _result(out, rows, cols, dtype):
    """The caller's output, checked, or a new one of a type; its row stride and kind."""
    if out is None:
        dtype = dtype or torch.bfloat16
        return _new((rows, cols), (cols, 1), dtype), cols, _out_kind(dtype)
    if tuple(out.shape) != (rows, cols) or not _here(out) or (out.stride(1) != 1 and cols > 1):
        raise ValueError(f"out must be a tensor [{rows}, {cols}] on the current CUDA device with unit column stride")
    return out, _ld(out), _out_kind(out.dtype)


def _opts(wait_limit_ns, inject_fault):
    if not wait_limit_ns and not inject_fault:
        return None
    return ctypes.byref(GemmOpts(wait_limit_ns, inject_fault, 0))


@dataclass
class Fp4Tensor:
    """A 4-bit tensor [rows, k]: packed codes [rows, ld >= ceil(k/2)] (ld a
    multiple of 16), scale bytes in tiles (one flat tensor, see the C header),
    and for FP4_NV the tensor's scale (None: 1)."""
    codes: torch.Tensor
    scale: torch.Tensor
    rows: int
    k: int
    kind: int
    tensor_scale: Optional[torch.Tensor] = None

    def ld(self) -> int:
        """Row stride of the codes, in bytes."""
        return self.codes.stride(0) if self.rows > 1 else _round16((self.k + 1) // 2)

    def buffers(self):
        """Address and row stride of the codes, address of the scale bytes, which
        have to hold what rows and k say."""
        c, s, rows, n = self.codes, self.scale, self.rows, (self.k + 1) // 2
        device = _cuda_device()
        if c.get_device() != device or s.get_device() != device:
            raise ValueError("a 4-bit tensor's codes and scale must be on the current CUDA device")
        shape, stride = c.shape, c.stride()
        if (len(shape) != 2 or shape[0] < rows or shape[1] < n or (stride[1] != 1 and n > 1) or
                c.itemsize != 1):
            raise ValueError(f"codes must be a byte tensor of [{rows}, at least {n}] with unit column stride")
        size = _scale_bytes(rows, self.k, self.kind)
        if s.numel() < size or s.itemsize != 1 or not s.is_contiguous():
            raise ValueError(f"scale must be a contiguous byte tensor of at least {size} elements")
        return c.data_ptr(), stride[0] if rows > 1 else _round16(n), s.data_ptr()

    def operand(self) -> _Fp4Operand:
        codes, ld, scale = self.buffers()
        return _Fp4Operand(codes, scale, _ts(self.tensor_scale), self.rows, self.k, ld, self.kind, 0)

    def scales(self) -> torch.Tensor:
        """The scale bytes as [rows, ceil(k / block)] (a copy)."""
        n = -(-self.k // FP4_BLOCK[self.kind])
        r, tiles = -(-self.rows // 128), -(-self.k // 256) * (4 if self.kind == FP4_NV else 2)
        t = self.scale.view(-1)[:r * tiles * 512].view(r, tiles, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, tiles * 4)
        return t[:self.rows, :n].contiguous()


def alloc_fp4(rows: int, k: int, kind: int, tensor_scale=None, device="cuda") -> Fp4Tensor:
    """Output buffers for fp4_quant (codes' rows padded to 16 bytes)."""
    codes = torch.empty((rows, (k + 31) // 32 * 16), dtype=torch.uint8, device=device)
    scale = torch.empty(_scale_bytes(rows, k, kind), dtype=torch.uint8, device=device)
    return Fp4Tensor(codes, scale, rows, k, kind, tensor_scale)


def _scale_bytes(rows, k, kind) -> int:
    """fp4_scale_bytes of the library."""
    return (rows + 127) // 128 * ((k + 255) // 256) * (2048 if kind == FP4_NV else 1024)


def _output(out, rows, k, kind, tensor_scale):
    """The caller's 4-bit output, checked, or a new one (alloc_fp4 on the current
    device), and what its buffers() returns."""
    if out is not None:
        if (out.rows, out.k, out.kind) != (rows, k, kind):
            raise ValueError(f"out must be a 4-bit tensor [{rows}, {k}] of kind {kind}")
        return out, out.buffers()
    ld = (k + 31) // 32 * 16
    codes = _new((rows, ld), (ld, 1), torch.uint8)
    scale = _new((_scale_bytes(rows, k, kind),), (1,), torch.uint8)
    return Fp4Tensor(codes, scale, rows, k, kind, tensor_scale), (codes.data_ptr(), ld, scale.data_ptr())


@_streamed
def fp4_tensor_scale(x, out=None):
    """The FP4_NV scale of a tensor: the smallest power of two t with
    amax <= 6 * 448 * t (1 for a tensor of zeros), on the device."""
    rows, cols, ld = _matrix(x)
    f = _fns()
    out = out if out is not None else _new((1,), (1,), torch.float32)
    n = f.fp4_tensor_scale_workspace()
    stream = _on(x)
    workspace = _scratch(n, x, stream)        # held until the call returns
    _check(f.fp4_tensor_scale(x.data_ptr(), rows, cols, ld, _ts(out), workspace.data_ptr(), n, stream), "fp4_tensor_scale")
    return out


_NONE = (None, 0, None)


@_streamed
def fp4_quant(x, kind: int = FP4_MX, tensor_scale=None, transpose: bool = False,
              out: Optional[Fp4Tensor] = None) -> Fp4Tensor:
    """BF16 [rows, cols] to 4 bits along the rows, or (transpose=True) along the
    columns, written as [cols, rows]."""
    shape = _matrix(x)
    rows, cols = (shape[1], shape[0]) if transpose else shape[:2]
    out, to = _output(out, rows, cols, kind, tensor_scale)
    both = _NONE + to if transpose else to + _NONE
    _check(_fns().fp4_quant(x.data_ptr(), *shape, kind, _ts(tensor_scale), *both, _on(x)), "fp4_quant")
    out.tensor_scale = tensor_scale
    return out


@_streamed
def fp4_quant_dual(x, kind: int = FP4_MX, tensor_scale=None, out: Optional[Fp4Tensor] = None,
                   out_t: Optional[Fp4Tensor] = None):
    """fp4_quant along the rows and along the columns from one read of x."""
    shape = _matrix(x)
    rows, cols = shape[:2]
    out, to = _output(out, rows, cols, kind, tensor_scale)
    out_t, to_t = _output(out_t, cols, rows, kind, tensor_scale)
    _check(_fns().fp4_quant(x.data_ptr(), *shape, kind, _ts(tensor_scale), *to, *to_t, _on(x)), "fp4_quant_dual")
    out.tensor_scale = out_t.tensor_scale = tensor_scale
    return out, out_t


@_streamed
def fp4_dequant(q: Fp4Tensor, out=None, out_dtype=None):
    """The values of a 4-bit tensor, [rows, k], BF16 or FP32."""
    op = q.operand()
    out, ld_out, kind = _result(out, q.rows, q.k, out_dtype)
    _check(_fns().fp4_dequant(ctypes.byref(op), out.data_ptr(), ld_out, kind, _on(out)), "fp4_dequant")
    return out


@_streamed
def fp4_gemm_scaled(a: Fp4Tensor, b: Fp4Tensor, out=None, out_dtype=None, accumulate: bool = False,
                    wait_limit_ns: int = 0, inject_fault: int = 0):
    """C = A B^T (or C += A B^T) on two 4-bit tensors of the same kind."""
    if out is None and accumulate:
        raise ValueError("accumulate needs out")
    oa, ob = a.operand(), b.operand()
    out, ld_out, kind = _result(out, a.rows, b.rows, out_dtype)
    _check(_fns().fp4_gemm_scaled(ctypes.byref(oa), ctypes.byref(ob), out.data_ptr(), ld_out, kind,
                                  1 if accumulate else 0, _opts(wait_limit_ns, inject_fault), _on(out)),
           "fp4_gemm_scaled")
    return out


@_streamed
def fp4_linear(x, w: Fp4Tensor, tensor_scale=None, out=None, out_dtype=None, workspace=None,
               wait_limit_ns: int = 0, inject_fault: int = 0):
    """y = x w^T: x [rows, k] BF16 is quantized like w and multiplied, in one
    call.  workspace: optional uint8 tensor of fp4_linear_workspace(...)
    bytes (allocated per call if None; up to 4 rows none is needed)."""
    rows, k, ld = _matrix(x)
    if k != w.k:
        raise ValueError(f"x has {k} columns, w {w.k}")
    ow = w.operand()
    out, ld_out, kind = _result(out, rows, w.rows, out_dtype)
    stream = _on(x)
    n = _linear_bytes(rows, k, w.kind)
    if n and workspace is None:
        workspace = _scratch(n, x, stream)
    elif n and not (_here(workspace) and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous tensor on the current CUDA device")
    _check(_fns().fp4_linear(x.data_ptr(), rows, ld, _ts(tensor_scale), ctypes.byref(ow),
                             out.data_ptr(), ld_out, kind,
                             workspace.data_ptr() if n else None, workspace.numel() if n else 0,
                             _opts(wait_limit_ns, inject_fault), stream), "fp4_linear")
    return out


def _linear_bytes(rows, k, kind) -> int:
    """fp4_linear_workspace of the library, which quantizes up to four rows in the
    product."""
    return 0 if rows <= 4 else rows * ((k + 31) // 32 * 16) + _scale_bytes(rows, k, kind)


_scratch_of = threading.local()
_SCRATCH = 1 << 20


def _scratch(n, x, stream):
    """n bytes on x's device for one call on `stream`.  Up to 1 MB they are kept
    for the next call of this thread on the stream (an allocation takes a
    third of such a call's time on the host); under stream capture, where the
    graph may outlive them, and above that they are allocated."""
    if n > _SCRATCH or torch._C._cuda_isCurrentStreamCapturing():
        return _new((n,), (1,), torch.uint8)      # x is on the current device
    kept = _scratch_of.__dict__
    key = (x.get_device(), stream)
    t = kept.get(key)
    if t is None:
        t = kept[key] = torch.empty(_SCRATCH, dtype=torch.uint8, device=x.device)
    return t


def fp4_linear_workspace(rows: int, k: int, kind: int) -> int:
    """Bytes of workspace that fp4_linear needs."""
    return int(_fns().fp4_linear_workspace(rows, k, kind))


# ------------------------------------------------- SwiGLU, 8-bit checkpoints
@dataclass
class SwigluCkpt:
    """gate and up [rows, cols] as FP8 with one UE8M0 scale per 128 columns."""
    gate: QTensor
    up: QTensor


def _groups(rows, cols, fmt):
    """[rows, cols] codes (rows padded to 16 bytes) and their 1x128 scales."""
    g = (cols + 127) // 128
    ls = _round4(g)
    return QTensor(_new((rows, cols), (_round16(cols), 1), torch.uint8),
                   _new((rows, ls), (ls, 1), torch.uint8), fmt, GRAN_1x128, g)


@_streamed
def fp8_swiglu_ckpt(gate, up, fmt: int = E4M3, fmt_h: int = E4M3, checkpoint: bool = True):
    """h = silu(gate) * up, quantized per 1x128 group (the down projection's A
    operand), and gate and up quantized the same way for the backward pass.
    gate and up may be the two halves of one tensor.  checkpoint=False
    (inference) writes h alone and returns (h, None)."""
    shape = rows, cols, ld_in = _matrix(gate, "gate")
    if _matrix(up, "up") != shape:
        raise ValueError("gate and up must have the same shape and row stride")
    ld = _round16(cols)
    h = _groups(rows, cols, fmt_h)
    ckpt, ptr, ls = None, (None, None, None, None), h.scale.shape[1]
    if checkpoint:
        g, u = _groups(rows, cols, fmt), _groups(rows, cols, fmt)
        ptr = (g.codes.data_ptr(), g.scale.data_ptr(), u.codes.data_ptr(), u.scale.data_ptr())
        ckpt = SwigluCkpt(g, u)
    _check(_fns().fp8_swiglu_ckpt(gate.data_ptr(), up.data_ptr(), rows, cols, ld_in, fmt_h,
                                  h.codes.data_ptr(), ld, h.scale.data_ptr(), ls, fmt, *ptr, ld, ls,
                                  _on(gate)), "fp8_swiglu_ckpt")
    return h, ckpt


def _half(q, rows, cols, device):
    """Addresses and row strides of a checkpoint half's codes and scales, which
    have to hold [rows, cols] and a byte per 128 columns."""
    c, s, groups = q.codes, q.scale, (cols + 127) // 128
    if c.get_device() != device or s.get_device() != device:
        raise ValueError("a checkpoint's codes and scales must be on the current CUDA device")
    if c.shape != (rows, cols):
        raise ValueError("dh and the checkpoint must have the same shape")
    ld, unit = c.stride()
    if c.itemsize != 1 or (unit != 1 and cols > 1):
        raise ValueError("a checkpoint's codes must be bytes with unit column stride")
    shape, stride = s.shape, s.stride()
    if (len(shape) != 2 or shape[0] < rows or shape[1] < groups or (stride[1] != 1 and groups > 1) or
            s.itemsize != 1):
        raise ValueError(f"a checkpoint's scales must be bytes [{rows}, at least {groups}] with unit column stride")
    return (c.data_ptr(), s.data_ptr(), ld, stride[0]) if rows > 1 else (c.data_ptr(), s.data_ptr(), _round16(cols),
                                                                         groups)


def _ckpt(c: SwigluCkpt, dh):
    """The checkpoint for the library; dh's rows, columns and row stride."""
    g, u = c.gate, c.up
    shape = rows, cols, _ = _matrix(dh, "dh")
    if g.gran != GRAN_1x128 or u.gran != GRAN_1x128 or g.fmt != u.fmt:
        raise ValueError("a checkpoint has 1x128 scales and one format")
    device = dh.get_device()
    gq, gs, ld, ls = _half(g, rows, cols, device)
    uq, us, ld_u, ls_u = _half(u, rows, cols, device)
    if ld != ld_u or ls != ls_u:
        raise ValueError("gate's and up's codes and scales must have the same strides")
    return _Ckpt(gq, gs, uq, us, rows, cols, ld, ls, g.fmt, 0), shape


@_streamed
def fp8_swiglu_ckpt_bwd(dh, ckpt: SwigluCkpt, out=None):
    """Gradients of gate and up from dh [rows, cols] and the checkpoint, BF16:
    one [rows, 2 cols] tensor, dgate in the first half, dup in the second."""
    c, (rows, cols, ld) = _ckpt(ckpt, dh)
    out, ld_out, kind = _result(out, rows, 2 * cols, torch.bfloat16)
    if kind != OUT_BF16:
        raise ValueError("out must be bfloat16")
    to = out.data_ptr()
    _check(_fns().fp8_swiglu_ckpt_bwd(dh.data_ptr(), ld, ctypes.byref(c), to, to + 2 * cols, ld_out, _on(dh)),
           "fp8_swiglu_ckpt_bwd")
    return out


@_streamed
def fp8_swiglu_ckpt_bwd_q(dh, ckpt: SwigluCkpt, fmt: int = E5M2, fmt_t: int = E5M2,
                          fmt_h: int = E4M3):
    """The gradients as FP8 operands: ([rows, 2 cols] per 1x128 group, dgate next
    to dup; the same transposed, [2 cols, rows], per 128 tokens; h rebuilt from
    the checkpoint and transposed, [cols, rows], per 128 tokens).  rows and cols
    must be multiples of 128."""
    c, (rows, cols, ld) = _ckpt(ckpt, dh)
    d = _groups(rows, 2 * cols, fmt)
    t = _groups(2 * cols, rows, fmt_t)
    h = _groups(cols, rows, fmt_h)
    dq, ds, tq, tl = d.codes.data_ptr(), d.scale.data_ptr(), t.codes.data_ptr(), t.scale.data_ptr()
    ld_qt, ld_st = t.codes.stride(0), t.scale.stride(0)
    g = _Grads(dq, dq + cols, ds, ds + cols // 128, tq, tq + cols * ld_qt, tl, tl + cols * ld_st,
               h.codes.data_ptr(), h.scale.data_ptr(), d.codes.stride(0), d.scale.stride(0), ld_qt,
               ld_st, fmt, fmt_t, fmt_h, 0)
    _check(_fns().fp8_swiglu_ckpt_bwd_q(dh.data_ptr(), ld, ctypes.byref(c), ctypes.byref(g), _on(dh)),
           "fp8_swiglu_ckpt_bwd_q")
    return d, t, h
