"""Layer norm, forward and backward, against 64 bits."""
import pathlib
import subprocess
import sys

import pytest
import torch

import adapt_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (1, 3584), (3, 7), (37, 16), (5, 33), (64, 128), (9, 500), (33, 513), (1000, 1536), (7, 4097),
         (333, 5001), (2, 8192), (3, 8193), (5, 20000)]


def values(rows, cols, dtype, seed=0, pad=0, shift=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed + rows * 131 + cols)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(1, cols + pad, generator=g, device="cuda"))
    return (x + shift).to(dtype)[:, pad:]


def params(cols, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed + cols)
    r = lambda: torch.randn(cols, generator=g, device="cuda")  # noqa: E731
    return (1 + 0.2 * r()).to(dtype), (0.1 * r()).to(dtype)


def check_stats(stats, mean, rstd, x):
    d = 40 * ref.U * x.double().abs().mean(1, keepdim=True)
    ref.close(stats[:, :1], mean, d + 1e-300, "mean")
    ref.close(stats[:, 1:], rstd, rstd * (d * rstd + 40 * ref.U), "rstd")


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("xt,yt,pt", [(BF16, BF16, F32), (F32, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16)])
def test_forward(cuda_lib, rows, cols, xt, yt, pt):
    x = values(rows, cols, xt)
    w, b = params(cols, pt)
    y, stats = cuda_lib.layernorm(x, w, b, 1e-5, out_dtype=yt)
    mean, rstd, want, tol = ref.norm(x, w, b, 1e-5)
    assert y.dtype == yt
    ref.close(y, want, tol + ref.half_step(yt) * want.abs() * 1.01 + 1e-38, "y")
    check_stats(stats, mean, rstd, x)


@pytest.mark.parametrize("pad", [1, 2, 8, 16, 37])
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", [(11, 1003), (6, 3584), (4, 9000), (70, 48)])
def test_strides(cuda_lib, rows, cols, xt, yt, pad):
    """Slices of wider tensors; what lies beside the output stays."""
    x = values(rows, cols, xt, pad=pad)
    whole = torch.full((rows + 2, cols + 2 * pad), 7.0, dtype=yt, device="cuda")
    out = whole[1:-1, pad:pad + cols]
    y, _ = cuda_lib.layernorm(x, out=out)
    assert y.data_ptr() == out.data_ptr()
    _, _, want, tol = ref.norm(x, None, None, 1e-5)
    ref.close(out, want, tol + ref.half_step(yt) * want.abs() * 1.01 + 1e-38, "y")
    whole[1:-1, pad:pad + cols] = 7.0
    assert (whole == 7.0).all()


@pytest.mark.parametrize("rows,cols,group", [(1, 3584, 0), (1000, 1536, 128), (37, 1003, 128), (37, 1003, 0), (3, 9001, 0),
                                             (3, 9001, 128), (130, 100, 128), (130, 100, 0), (2, 1, 0)])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("with_y", [False, True])
def test_fp8(cuda_lib, rows, cols, group, fmt, with_y):
    x = values(rows, cols, BF16, seed=fmt)
    w, b = params(cols, F32)
    q, y, stats = cuda_lib.fp8_layernorm(x, w, b, 1e-5, group=group, fmt=fmt, with_y=with_y)
    mean, rstd, want, tol = ref.norm(x, w, b, 1e-5)
    check_stats(stats, mean, rstd, x)
    if with_y:
        ref.close(y, want, tol + ref.half_step(BF16) * want.abs() * 1.01, "y")
    e, moved, tol = ref.fp8_groups(want, tol, group, fmt)
    byte = q.scales().int() - 127
    assert ((byte == e) | moved).all()
    width = group or cols
    values_of = q.codes.view((torch.float8_e4m3fn, torch.float8_e5m2)[fmt]).double()
    got = values_of * torch.exp2(byte.double()).repeat_interleave(width, 1)[:, :cols]
    ref.close(got, want, tol, "codes")


MANY = [(5200, 96), (5200, 301), (1300, 1027), (2500, 2051), (2500, 3584), (700, 5001), (700, 8191)]


@pytest.mark.parametrize("rows,cols", MANY)
@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("pad", [0, 3])
def test_many_rows(cuda_lib, rows, cols, xt, yt, pad):
    """Many rows a CTA, whole tensors and slices."""
    if pad:
        test_strides(cuda_lib, rows, cols, xt, yt, pad)
    else:
        test_forward(cuda_lib, rows, cols, xt, yt, F32)


@pytest.mark.parametrize("rows,cols", MANY)
@pytest.mark.parametrize("group", [0, 128])
def test_fp8_of_many_rows(cuda_lib, rows, cols, group):
    test_fp8(cuda_lib, rows, cols, group, 0, True)


def test_fp8_feeds_the_product(cuda_lib):
    """The codes are an operand of the FP8 product, as fp8_quant_token's are."""
    x = values(256, 512, BF16)
    w, b = params(512, F32)
    g = torch.Generator(device="cuda").manual_seed(5)
    weight = torch.randn(256, 512, generator=g, device="cuda").bfloat16()
    wq = cuda_lib.fp8_quant_block128(weight)
    _, _, y, _ = ref.norm(x, w, b, 1e-5)
    wv = wq.codes.view(torch.float8_e4m3fn).double() * torch.exp2(wq.scales().double() - 127).repeat_interleave(128, 0).repeat_interleave(128, 1)
    want = y @ wv.t()
    # a code is off by at most 2^-4 of its value, or by half of the smallest step of its scale
    for group in (0, 128):
        q, _, _ = cuda_lib.fp8_layernorm(x, w, b, 1e-5, group=group)
        got = cuda_lib.fp8_gemm_scaled(cuda_lib.FPROP, q, wq, out_dtype=F32)
        step = torch.exp2(q.scales().double() - 127 - 10).repeat_interleave(group or 512, 1)
        ref.close(got, want, (y.abs() * 2.0 ** -4 + step) @ wv.abs().t() * 1.01, "product")
    assert cuda_lib.fp8hg_get_device_error() == 0


def test_far_from_zero(cuda_lib):
    """A row whose values are 10^4 times its spread apart from zero."""
    x = values(40, 3000, F32, shift=0.0) + 1e4
    y, stats = cuda_lib.layernorm(x)
    mean, rstd, want, tol = ref.norm(x, None, None, 1e-5)
    ref.close(y, want, tol, "y")
    check_stats(stats, mean, rstd, x)


def test_constant_and_non_finite_rows(cuda_lib):
    x = values(6, 300, F32)
    x[1] = 3.0                       # no spread: the bias alone
    x[2, 5] = float("nan")
    x[4, 299] = float("inf")
    w, b = params(300, F32)
    y, _ = cuda_lib.layernorm(x, w, b)
    assert torch.equal(y[1], b)
    assert y[2].isnan().all() and y[4].isnan().all()
    _, _, want, tol = ref.norm(x, w, b, 1e-5)
    for i in (0, 3, 5):
        ref.close(y[i], want[i], tol[i] + ref.U * want[i].abs(), "y")
    q, _, _ = cuda_lib.fp8_layernorm(x, w, b, group=128)
    assert (q.scales()[2] == 255).all() and (q.codes[2] == 0x7F).all() and (q.scales()[[0, 1, 3, 5]] != 255).all()


def test_in_place_and_empty(cuda_lib):
    x = values(30, 700, BF16)
    want, _ = cuda_lib.layernorm(x)
    got, _ = cuda_lib.layernorm(x, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
    for shape in ((0, 5), (5, 0)):
        y, stats = cuda_lib.layernorm(torch.empty(shape, dtype=BF16, device="cuda"))
        assert y.shape == shape and stats.shape == (shape[0], 2)


@pytest.mark.parametrize("rows,cols", SIZES + [(2500, 300), (900, 64)])
@pytest.mark.parametrize("xt,dt,pt", [(BF16, BF16, F32), (F32, BF16, F32), (F32, F32, BF16), (BF16, F32, None)])
@pytest.mark.parametrize("with_add", [False, True])
def test_backward(cuda_lib, rows, cols, xt, dt, pt, with_add):
    x, dy = values(rows, cols, xt), values(rows, cols, dt, seed=3, shift=0.01)
    w = None if pt is None else params(cols, pt)[0]
    add = values(rows, cols, xt, seed=4) if with_add else None
    _, stats = cuda_lib.layernorm(x, w)
    dx, dw, db = cuda_lib.layernorm_bwd(dy, x, w, stats, add=add)
    for got, (want, tol), t, what in zip((dx, dw, db), ref.norm_bwd(dy, x, w, stats, add), (xt, F32, F32), ("dx", "dw", "db")):
        assert got.dtype == t
        ref.close(got, want, tol + ref.half_step(t) * want.abs() * 1.01 + 1e-37, what)
    only, none, _ = cuda_lib.layernorm_bwd(dy, x, w, stats, add=add, params=False)
    assert torch.equal(only, dx) and none is None


@pytest.mark.parametrize("rows,cols", [(2100, 5001), (2050, 4104), (2048, 5120), (2500, 301), (700, 5123), (1300, 1027)])
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("with_add", [False, True])
def test_backward_of_many_rows(cuda_lib, rows, cols, kind, with_add):
    """Many rows a CTA, even and odd ones, all of one type."""
    x, dy = values(rows, cols, kind), values(rows, cols, kind, seed=3, shift=0.01)
    w = params(cols, BF16)[0]
    add = values(rows, cols, kind, seed=4) if with_add else None
    _, stats = cuda_lib.layernorm(x, w)
    for got, (want, tol), t, what in zip(cuda_lib.layernorm_bwd(dy, x, w, stats, add=add), ref.norm_bwd(dy, x, w, stats, add), (kind, F32, F32),
                                         ("dx", "dw", "db")):
        ref.close(got, want, tol + ref.half_step(t) * want.abs() * 1.01 + 1e-37, what)


@pytest.mark.parametrize("pad", [1, 4, 8, 16, 37])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_backward_strides(cuda_lib, xt, pad):
    rows, cols = 19, 1003
    x, dy = values(rows, cols, xt, pad=pad), values(rows, cols, BF16, seed=3, pad=pad + 1)
    _, stats = cuda_lib.layernorm(x)
    whole = torch.full((rows, cols + 2 * pad), 7.0, dtype=xt, device="cuda")
    dx, dw, db = cuda_lib.layernorm_bwd(dy, x, None, stats, out=whole[:, pad:pad + cols])
    for got, (want, tol), t in zip((dx, dw, db), ref.norm_bwd(dy, x, None, stats, None), (xt, F32, F32)):
        ref.close(got, want, tol + ref.half_step(t) * want.abs() * 1.01 + 1e-37, "gradient")
    whole[:, pad:pad + cols] = 7.0
    assert (whole == 7.0).all()


def test_backward_in_place_and_empty(cuda_lib):
    x, dy, add = values(30, 700, BF16), values(30, 700, BF16, seed=2), values(30, 700, BF16, seed=4)
    _, stats = cuda_lib.layernorm(x)
    want, _, _ = cuda_lib.layernorm_bwd(dy, x, None, stats, add=add)
    got, _, _ = cuda_lib.layernorm_bwd(dy, x, None, stats, add=add, out=add)
    assert got.data_ptr() == add.data_ptr() and torch.equal(got, want)
    empty = torch.empty(0, 9, dtype=BF16, device="cuda")
    dx, dw, db = cuda_lib.layernorm_bwd(empty, empty, None, torch.empty(0, 2, device="cuda"))
    assert dx.shape == (0, 9) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("cols", [300, 4104, 5001, 8200])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_in_place(cuda_lib, cols, kind):
    """y over x; dx over dy and over x, with dw and db from what was there."""
    x, dy = values(700, cols, kind), values(700, cols, kind, seed=2)
    w, b = params(cols, F32)
    y, stats = cuda_lib.layernorm(x, w, b)
    over = x.clone()
    assert torch.equal(cuda_lib.layernorm(over, w, b, out=over)[0], y)
    want = cuda_lib.layernorm_bwd(dy, x, w, stats)
    over = dy.clone()
    assert all(torch.equal(p, q) for p, q in zip(cuda_lib.layernorm_bwd(over, x, w, stats, out=over), want))
    over = x.clone()
    assert all(torch.equal(p, q) for p, q in zip(cuda_lib.layernorm_bwd(dy, over, w, stats, out=over), want))


def test_every_width_in_a_new_process(cuda_lib):
    """A kernel's first call in a process asks for what its shared memory takes, whatever
    its width: from narrow to wide, so that no wider one came before."""
    code = """
import torch
import fp8_hybrid_granularity_gb300 as lib
for cols in range(256, 8193, 256):
    for kind in (torch.bfloat16, torch.float32):
        for rows in (2, 5000):
            for n in (cols - 1, cols):
                x = torch.ones(rows, n, dtype=kind, device="cuda")
                y, stats = lib.layernorm(x)
                assert (y == 0).all(), (rows, n, kind)
                if kind == torch.bfloat16:
                    lib.fp8_layernorm(x)
                dx, dw, db = lib.layernorm_bwd(x, x, None, stats)
                assert (db == rows).all(), (rows, n, kind)
                lib.layernorm_bwd(x, x, None, stats, add=x)
torch.cuda.synchronize()
"""
    root = pathlib.Path(__file__).resolve().parent.parent
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_gradient_by_differences(cuda_lib):
    """The backward call against differences of the forward call's sum(y * c)."""
    rows, cols, h = 4, 24, 2.0 ** -6
    x, c = values(rows, cols, F32), values(rows, cols, F32, seed=9)
    w, b = params(cols, F32)
    _, stats = cuda_lib.layernorm(x, w, b)
    dx, dw, db = cuda_lib.layernorm_bwd(c, x, w, stats)

    def f(x, w, b):
        return (ref.norm(x, w, b, 1e-5)[2] * c.double()).sum()

    for t, got in ((x, dx), (w, dw), (b, db)):
        for i in (0, 7, cols - 1, t.numel() - 1):
            d = torch.zeros(t.numel(), dtype=torch.float64, device="cuda")
            d[i] = h
            d = d.view(t.shape)
            up, down = ([(p.double() + s * d) if p is t else p for p in (x, w, b)] for s in (1, -1))
            want = (f(*up) - f(*down)) / (2 * h)
            # third derivatives are below 20 here: h^2 / 6 of them
            assert abs(float(got.flatten()[i]) - float(want)) < 20 * h * h, (i, float(got.flatten()[i]), float(want))


def test_captured(cuda_lib):
    """A graph replays with new inputs; its workspace is its own."""
    x, dy = values(300, 1000, BF16), values(300, 1000, BF16, seed=2)
    w, b = params(1000, F32)
    cuda_lib.layernorm_bwd(dy, x, w, cuda_lib.layernorm(x, w, b)[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, stats = cuda_lib.layernorm(x, w, b)
        dx, dw, db = cuda_lib.layernorm_bwd(dy, x, w, stats)
    x2, dy2 = values(300, 1000, BF16, seed=7), values(300, 1000, BF16, seed=8)
    x.copy_(x2), dy.copy_(dy2)
    graph.replay()
    # other calls of this thread between replays do not touch what the graph holds
    want, st = cuda_lib.layernorm(x2, w, b)
    again = cuda_lib.layernorm_bwd(dy2, x2, w, st)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


def test_other_stream(cuda_lib):
    x = values(500, 2000, BF16)
    w, b = params(2000, F32)
    want, stats = cuda_lib.layernorm(x, w, b)
    grads = cuda_lib.layernorm_bwd(x, x, w, stats)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, st = cuda_lib.layernorm(x, w, b, stream=s)
    got = cuda_lib.layernorm_bwd(x, x, w, st, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip(got, grads))
