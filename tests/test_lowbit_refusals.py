"""The Python side of the 4-bit and SwiGLU calls without a GPU: which stream a
handle names, and what is refused before anything reaches the library.  Tensors
on a GPU are stood in for; no call here launches anything."""
import contextlib

import pytest
import torch

import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import lowbit


def test_stream_handles(monkeypatch):
    """A torch stream as it is, a raw handle wrapped, and handle 0 as the
    default stream (a wrapper around 0 would be a new stream)."""
    entered = []

    class Stream:
        pass

    @contextlib.contextmanager
    def enter(s):
        entered.append(s)
        yield

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda: "default")
    call = lowbit._streamed(lambda v, w=0: v + w)
    own = Stream()
    assert call(1, w=2) == 3 and entered == []
    assert call(1, w=2, stream=own) == 3 and call(2, stream=0x5000) == 2 and call(3, stream=0) == 3
    assert entered == [own, ("external", 0x5000), "default"]


class StandIn:
    """A tensor that says it is on GPU `device`; its memory, never used, is the
    CPU's."""

    def __init__(self, t, device=0):
        self._t, self._device = t, device
        self.dtype, self.shape = t.dtype, t.shape
        self.is_cuda, self.device = True, torch.device("cuda", device)

    def get_device(self):
        return self._device

    def __getattr__(self, name):
        return getattr(self._t, name)


class Reached(Exception):
    """The library was called."""


@pytest.fixture
def gpu0(monkeypatch):
    """GPU 0 is current; the library only says that it was reached."""
    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_workspace"):
                    return 4096
                raise Reached(name)
            return call

    monkeypatch.setattr(lowbit, "_cuda_device", lambda: 0)
    monkeypatch.setattr(lowbit, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(lowbit, "_fns", Library)
    # what the calls allocate is on GPU 0 too
    monkeypatch.setattr(lowbit, "_new", lambda *a: StandIn(torch.empty_strided(*a[:2], dtype=a[2])), raising=False)
    monkeypatch.setattr(lowbit, "_scratch", lambda n, x, stream: StandIn(torch.empty(n, dtype=torch.uint8)))
    return lambda t: StandIn(t)


def bf16(rows, cols):
    return torch.zeros(rows, cols, dtype=torch.bfloat16)


def fp4(on, rows=40, k=64, kind=fp8hg.FP4_MX, ts=None):
    q = fp8hg.alloc_fp4(rows, k, kind, ts, device="cpu")
    q.codes, q.scale = on(q.codes), on(q.scale)
    return q


def ckpt(on, rows=4, cols=128):
    half = lambda: fp8hg.QTensor(on(torch.zeros(rows, cols, dtype=torch.uint8)),
                                 on(torch.zeros(rows, (cols + 511) // 512 * 4, dtype=torch.uint8)), fp8hg.E4M3,
                                 fp8hg.GRAN_1x128, (cols + 127) // 128)
    return fp8hg.SwigluCkpt(half(), half())


def f32(*shape):
    return torch.zeros(shape)


# every tensor argument of every call: name -> the call with one argument from `one`, the others from `on`
CALLS = {
    "tensor_scale x": lambda on, one: fp8hg.fp4_tensor_scale(one(bf16(4, 64))),
    "tensor_scale out": lambda on, one: fp8hg.fp4_tensor_scale(on(bf16(4, 64)), out=one(f32(1))),
    "quant x": lambda on, one: fp8hg.fp4_quant(one(bf16(4, 64))),
    "quant scale": lambda on, one: fp8hg.fp4_quant(on(bf16(4, 64)), fp8hg.FP4_NV, one(f32(1))),
    "quant out": lambda on, one: fp8hg.fp4_quant(on(bf16(40, 64)), out=fp4(one)),
    "quant transposed out": lambda on, one: fp8hg.fp4_quant(on(bf16(64, 40)), transpose=True, out=fp4(one)),
    "dual x": lambda on, one: fp8hg.fp4_quant_dual(one(bf16(40, 64))),
    "dual out": lambda on, one: fp8hg.fp4_quant_dual(on(bf16(40, 64)), out=fp4(one)),
    "dual out_t": lambda on, one: fp8hg.fp4_quant_dual(on(bf16(40, 64)), out_t=fp4(one, 64, 40)),
    "dequant q": lambda on, one: fp8hg.fp4_dequant(fp4(one)),
    "dequant out": lambda on, one: fp8hg.fp4_dequant(fp4(on), out=one(bf16(40, 64))),
    "gemm a": lambda on, one: fp8hg.fp4_gemm_scaled(fp4(one), fp4(on)),
    "gemm b": lambda on, one: fp8hg.fp4_gemm_scaled(fp4(on), fp4(one)),
    "gemm scale": lambda on, one: fp8hg.fp4_gemm_scaled(fp4(on, kind=fp8hg.FP4_NV, ts=one(f32(1))),
                                                        fp4(on, kind=fp8hg.FP4_NV)),
    "gemm out": lambda on, one: fp8hg.fp4_gemm_scaled(fp4(on), fp4(on), out=one(bf16(40, 40))),
    "linear x": lambda on, one: fp8hg.fp4_linear(one(bf16(8, 64)), fp4(on)),
    "linear w": lambda on, one: fp8hg.fp4_linear(on(bf16(8, 64)), fp4(one)),
    "linear out": lambda on, one: fp8hg.fp4_linear(on(bf16(8, 64)), fp4(on), out=one(bf16(8, 40))),
    "linear workspace": lambda on, one: fp8hg.fp4_linear(on(bf16(8, 64)), fp4(on),
                                                         workspace=one(torch.zeros(2048, dtype=torch.uint8))),
    "swiglu gate": lambda on, one: fp8hg.fp8_swiglu_ckpt(one(bf16(4, 128)), on(bf16(4, 128))),
    "swiglu up": lambda on, one: fp8hg.fp8_swiglu_ckpt(on(bf16(4, 128)), one(bf16(4, 128))),
    "bwd dh": lambda on, one: fp8hg.fp8_swiglu_ckpt_bwd(one(bf16(4, 128)), ckpt(on)),
    "bwd checkpoint": lambda on, one: fp8hg.fp8_swiglu_ckpt_bwd(on(bf16(4, 128)), ckpt(one)),
    "bwd out": lambda on, one: fp8hg.fp8_swiglu_ckpt_bwd(on(bf16(4, 128)), ckpt(on), out=one(bf16(4, 256))),
    "bwd_q dh": lambda on, one: fp8hg.fp8_swiglu_ckpt_bwd_q(one(bf16(128, 128)), ckpt(on, 128)),
    "bwd_q checkpoint": lambda on, one: fp8hg.fp8_swiglu_ckpt_bwd_q(on(bf16(128, 128)), ckpt(one, 128)),
}


@pytest.mark.parametrize("name", CALLS)
def test_tensors_elsewhere_are_refused(gpu0, name):
    """A call launches on the current device: tensors of another GPU, or of
    the CPU, never reach it."""
    with pytest.raises(Reached):
        CALLS[name](gpu0, gpu0)
    for elsewhere in (lambda t: StandIn(t, 1), lambda t: t):
        with pytest.raises(ValueError):
            CALLS[name](gpu0, elsewhere)


# a 4-bit tensor of 130 rows of 300, and ways in which its buffers hold less than that
FP4_CALLS = {
    "quant out": lambda q: fp8hg.fp4_quant(StandIn(bf16(130, 300)), q.kind, out=q),
    "quant transposed out": lambda q: fp8hg.fp4_quant(StandIn(bf16(300, 130)), q.kind, transpose=True, out=q),
    "dual out": lambda q: fp8hg.fp4_quant_dual(StandIn(bf16(130, 300)), q.kind, out=q),
    "dual out_t": lambda q: fp8hg.fp4_quant_dual(StandIn(bf16(300, 130)), q.kind, out_t=q),
    "dequant": lambda q: fp8hg.fp4_dequant(q),
    "gemm a": lambda q: fp8hg.fp4_gemm_scaled(q, fp4(StandIn, 8, 300, q.kind)),
    "gemm b": lambda q: fp8hg.fp4_gemm_scaled(fp4(StandIn, 8, 300, q.kind), q),
    "linear w": lambda q: fp8hg.fp4_linear(StandIn(bf16(2, 300)), q),
}


def broken(field, value):
    def change(q):
        setattr(q, field, StandIn(value))
    return change


def buffers_that_do_not_hold(kind):
    n = fp8hg.alloc_fp4(130, 300, kind, device="cpu").scale.numel()
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    return {
        "codes with a row too few": broken("codes", u8(129, 160)),
        "codes with a byte too few a row": broken("codes", u8(130, 160)[:, :149]),
        "codes of another type": broken("codes", torch.zeros(130, 160, dtype=torch.int16)),
        "codes of every second byte": broken("codes", u8(130, 320)[:, ::2]),
        "flat codes": broken("codes", u8(130 * 160)),
        "scale with a byte too few": broken("scale", u8(n - 1)),
        "scale of 128 rows": broken("scale", u8(n // 2)),
        "scale of every second byte": broken("scale", u8(2 * n)[::2]),
        "scale of another type": broken("scale", torch.zeros(n)),
    }


@pytest.mark.parametrize("kind", [fp8hg.FP4_MX, fp8hg.FP4_NV])
@pytest.mark.parametrize("name", FP4_CALLS)
def test_buffers_that_do_not_hold_the_tensor(gpu0, name, kind):
    """A 4-bit tensor whose codes or scale bytes hold less than rows and k say
    is refused: a kernel would read or write past them."""
    with pytest.raises(Reached):
        FP4_CALLS[name](fp4(gpu0, 130, 300, kind))
    # more than the tensor needs, and one-byte types other than uint8, are as good
    q = fp4(gpu0, 130, 300, kind)
    broken("codes", torch.zeros(200, 176, dtype=torch.int8))(q)
    broken("scale", torch.zeros(8, 2048, dtype=torch.uint8))(q)
    with pytest.raises(Reached):
        FP4_CALLS[name](q)
    for what, change in buffers_that_do_not_hold(kind).items():
        q = fp4(gpu0, 130, 300, kind)
        change(q)
        with pytest.raises(ValueError):
            FP4_CALLS[name](q)
            pytest.fail(what)


def test_workspace_with_gaps(gpu0):
    with pytest.raises(ValueError):
        fp8hg.fp4_linear(gpu0(bf16(8, 64)), fp4(gpu0), workspace=gpu0(torch.zeros(8192, dtype=torch.uint8)[::2]))


CKPT_CALLS = {
    "bwd": lambda c: fp8hg.fp8_swiglu_ckpt_bwd(StandIn(bf16(128, 640)), c),
    "bwd_q": lambda c: fp8hg.fp8_swiglu_ckpt_bwd_q(StandIn(bf16(128, 640)), c),
}


@pytest.mark.parametrize("name", CKPT_CALLS)
@pytest.mark.parametrize("half", ["gate", "up"])
def test_checkpoint_buffers_that_do_not_hold_it(gpu0, name, half):
    """[128, 640] codes and [128, 5 of 8] scale bytes, and ways to hold less."""
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)
    with pytest.raises(Reached):
        CKPT_CALLS[name](ckpt(gpu0, 128, 640))
    for field, value in (("codes", u8(128, 1280)[:, ::2]), ("codes", torch.zeros(128, 640, dtype=torch.int16)),
                         ("scale", u8(127, 8)), ("scale", u8(128, 8)[:, :4]), ("scale", u8(128, 16)[:, ::2]),
                         ("scale", u8(128 * 8)), ("scale", torch.zeros(128, 8))):
        c = ckpt(gpu0, 128, 640)
        setattr(getattr(c, half), field, gpu0(value))
        with pytest.raises(ValueError):
            CKPT_CALLS[name](c)
            pytest.fail(f"{field} {tuple(value.shape)} {value.dtype}")


def row(n, stride, dtype=torch.bfloat16):
    """One row of n elements with a row stride that says nothing."""
    return torch.zeros(2 * (n + stride), dtype=dtype).as_strided((1, n), (stride, 1))


@pytest.mark.parametrize("stride", [0, 1, 99, 129, 4096])
def test_strides_of_one_row_say_nothing(gpu0, stride):
    """Operands of one row are taken with any row stride, also unlike each other's."""
    for call in (lambda: fp8hg.fp8_swiglu_ckpt(gpu0(row(128, stride)), gpu0(bf16(1, 128))),
                 lambda: fp8hg.fp8_swiglu_ckpt(gpu0(bf16(1, 128)), gpu0(row(128, stride))),
                 lambda: fp8hg.fp4_linear(gpu0(row(64, stride)), fp4(gpu0))):
        with pytest.raises(Reached):
            call()
    assert lowbit._matrix(gpu0(row(100, stride))) == (1, 100, 112) and lowbit._ld(gpu0(row(100, stride))) == 112
    q = fp4(gpu0, 1, 100)
    broken("codes", row(64, stride, torch.uint8))(q)
    assert q.ld() == 64 and q.buffers()[1] == 64
    c = ckpt(gpu0, 1, 128)
    c.gate.codes, c.up.scale = gpu0(row(128, stride, torch.uint8)), gpu0(row(4, stride, torch.uint8))
    with pytest.raises(Reached):
        fp8hg.fp8_swiglu_ckpt_bwd(gpu0(row(128, stride)), c)
    native = lowbit._ckpt(c, gpu0(row(128, stride)))[0]
    assert (native.ld_q, native.ld_s) == (128, 1)


def test_rows_of_the_quantizer_along_the_columns():
    """One row more than its grid holds is refused before the launch."""
    fake, rows = 0x10000, 32767 * 256 + 1
    call = lowbit._fns().fp4_quant
    assert call(fake, rows, 32, 32, fp8hg.FP4_MX, None, None, 0, None, fake, 2 ** 22, fake, None) == 3
    assert call(fake, rows, 32, 32, fp8hg.FP4_MX, None, fake, 16, fake, fake, 2 ** 22, fake, None) == 3


def test_scale_views():
    """QTensor.scales() is the unpadded slice: of whatever holds the scales, and
    of no more columns than there are."""
    import numpy as np
    for s in (torch.arange(32, dtype=torch.uint8).reshape(4, 8), np.arange(32, dtype=np.uint8).reshape(4, 8)):
        for n in (0, 5, 8, 9):
            got = fp8hg.QTensor(None, s, fp8hg.E4M3, fp8hg.GRAN_1x128, n).scales()
            assert tuple(got.shape) == (4, min(n, 8)) and (got == s[:, :n]).all()
            got[...] = 7                    # a view
            assert (s[:, :n] == 7).all()


@pytest.mark.parametrize("kind,block", [(fp8hg.FP4_MX, 32), (fp8hg.FP4_NV, 16)])
@pytest.mark.parametrize("rows,k", [(0, 64), (5, 0), (0, 0), (5, 70), (129, 257)])
def test_fp4_scales_of_any_size(kind, block, rows, k):
    """Fp4Tensor.scales() of empty tensors, and from scale arrays larger than the tensor needs."""
    q = fp8hg.alloc_fp4(rows, k, kind, device="cpu")
    q.scale.copy_(torch.arange(q.scale.numel()) % 251)
    want = q.scales()
    assert want.shape == (rows, -(-k // block)) and want.dtype == torch.uint8
    tiles = -(-k // 256) * 256 // block // 4
    for r, j in ((0, 0), (rows - 1, want.shape[1] - 1)):
        if want.numel():
            at = ((r // 128) * tiles + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4
            assert want[r, j] == q.scale[at]
    q.scale = torch.cat((q.scale, torch.zeros(777, dtype=torch.uint8)))
    assert torch.equal(q.scales(), want)


def test_refused_calls_change_nothing(monkeypatch, gpu0):
    """The outputs given to a call that the library refuses keep their tensor scale."""
    class Library:
        def fp4_quant(self, *args):
            return 1

    monkeypatch.setattr(lowbit, "_fns", Library)
    old, new = gpu0(f32(1)), gpu0(f32(1))
    q, qt = (fp4(gpu0, *shape, fp8hg.FP4_NV, old) for shape in ((40, 64), (64, 40)))
    for call in (lambda: fp8hg.fp4_quant(gpu0(bf16(40, 64)), fp8hg.FP4_NV, new, out=q),
                 lambda: fp8hg.fp4_quant(gpu0(bf16(64, 40)), fp8hg.FP4_NV, new, transpose=True, out=q),
                 lambda: fp8hg.fp4_quant_dual(gpu0(bf16(40, 64)), fp8hg.FP4_NV, new, out=q, out_t=qt)):
        with pytest.raises(fp8hg.Fp8hgError):
            call()
        assert q.tensor_scale is old and qt.tensor_scale is old


@pytest.mark.parametrize("kind", [fp8hg.FP4_MX, fp8hg.FP4_NV])
def test_linear_scratch_is_what_the_library_needs(kind):
    """Rows that the product quantizes itself need none: one rule for both sides."""
    for rows in list(range(12)) + [127, 128, 129, 1000]:
        for k in (1, 64, 257, 3584):
            assert lowbit._linear_bytes(rows, k, kind) == lowbit._fns().fp4_linear_workspace(rows, k, kind)
