"""Layer norm at the edges of what a call may be given: rows whose sums are exact, so
that mean and rstd have one right value, and offsets past 32 bits."""
import pytest
import torch

import adapt_ref as ref
from test_gpu_layernorm import check_stats, params, values

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("rows,cols", [(7, 1), (40, 3), (33, 127), (5, 1003), (4100, 49), (3000, 771), (2500, 3583), (700, 5001), (9, 8192),
                                       (5, 20000)])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_exact_sums(cuda_lib, rows, cols, kind):
    """Small whole numbers: the sums are exact in FP32, the mean is their quotient, correctly
    rounded; of rows with a mean of zero, rstd is that of the correctly rounded variance
    (rounded once, like the quotient: a double's rounding moves neither, its 53 bits being
    more than twice 24 and two)."""
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda")
    _, stats = cuda_lib.layernorm(x.to(kind))
    assert torch.equal(stats[:, 0], (x.sum(1).double() / cols).float())
    x[:, cols // 2:2 * (cols // 2)] = -x[:, :cols // 2]
    x[:, 2 * (cols // 2):] = 0
    x[:, 0] += (x == 0).all(1) & (cols > 1)
    x[:, cols // 2] -= (x[:, 0] + x[:, cols // 2]) * (cols > 1)
    assert (x.sum(1) == 0).all()
    _, stats = cuda_lib.layernorm(x.to(kind), eps=2.0 ** -40)
    var = (x * x).sum(1).double() / cols
    want = (var.float() + 2.0 ** -40).double().rsqrt()
    half = torch.exp2(torch.frexp(want)[1].double() - 25)
    assert (stats[:, 0] == 0).all() and ((stats[:, 1].double() - want).abs() <= half * (1 + 1e-6)).all()


def check(cuda_lib, x, dy, y, stats, dx, rows, w, b):
    """Some rows of the results."""
    x, dy, y, stats, dx = (t[rows] for t in (x, dy, y, stats, dx))
    mean, rstd, want, tol = ref.norm(x, w, b, 1e-5)
    check_stats(stats, mean, rstd, x)
    ref.close(y, want, tol + ref.half_step(y.dtype) * want.abs() * 1.01, "y")
    want, tol = ref.norm_bwd(dy, x, w, stats, None)[0]
    ref.close(dx, want, tol + ref.half_step(dx.dtype) * want.abs() * 1.01 + 1e-37, "dx")


@pytest.mark.parametrize("cols", [1003, 3584, 9001])
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("at", [16, 5])
def test_rows_far_apart(cuda_lib, cols, kind, at):
    """Row offsets that pass 2^31 elements: x, dy, y and dx slices of one wide buffer."""
    rows = 6
    width = (1 << 29) + (0 if at == 16 else 3)
    buf = torch.empty(rows, width, dtype=kind, device="cuda")
    x, dy, y, dx = (buf[:, at + 16384 * i:at + 16384 * i + cols] for i in range(4))
    x.copy_(values(rows, cols, kind)), dy.copy_(values(rows, cols, kind, seed=3))
    w, b = params(cols, F32)
    _, stats = cuda_lib.layernorm(x, w, b, out=y)
    _, dw, db = cuda_lib.layernorm_bwd(dy, x, w, stats, out=dx)
    check(cuda_lib, x, dy, y, stats, dx, torch.arange(rows, device="cuda"), w, b)
    for got, (want, tol) in zip((dw, db), ref.norm_bwd(dy, x, w, stats, None)[1:]):
        ref.close(got, want, tol + ref.U * want.abs(), "gradient")


@pytest.mark.parametrize("rows,cols", [(600_000, 3600), (262_200, 8200)])
def test_more_than_2_to_31_elements(cuda_lib, rows, cols):
    x = torch.randn(rows, cols, device="cuda", dtype=BF16)
    dy = torch.randn(rows, cols, device="cuda", dtype=BF16)
    assert x.numel() > 1 << 31
    w, b = params(cols, F32)
    q, y, stats = cuda_lib.fp8_layernorm(x, w, b, 1e-5, with_y=True)
    dx, dw, db = cuda_lib.layernorm_bwd(dy, x, w, stats)
    sel = torch.cat([torch.arange(0, rows, rows // 50, device="cuda"), torch.arange(rows - 20, rows, device="cuda"),
                     (1 << 31) // cols + torch.arange(-3, 4, device="cuda")])
    check(cuda_lib, x, dy, y, stats, dx, sel, w, b)
    _, _, want, tol = ref.norm(x[sel], w, b, 1e-5)
    e, moved, tol = ref.fp8_groups(want, tol, 0, 0)
    byte = q.scales()[sel].int() - 127
    assert ((byte == e) | moved).all()
    ref.close(q.codes[sel].view(torch.float8_e4m3fn).double() * torch.exp2(byte.double()), want, tol, "codes")
    # some columns of the sums over the rows, each within the bound of its own magnitudes
    for c in (0, cols // 2, cols - 1):
        d, xh = dy[:, c].double(), (x[:, c].double() - stats[:, 0].double()) * stats[:, 1].double()
        steps = (rows / 64 + 60) * ref.U
        assert abs(float(db[c]) - float(d.sum())) <= steps * float(d.abs().sum())
        assert abs(float(dw[c]) - float((d * xh).sum())) <= (steps + 8 * ref.U) * float((d.abs() * (xh.abs() + 1)).sum())


@pytest.mark.parametrize("rows,cols", [(16384, 3584), (700, 5001), (9, 20000)])
def test_the_same_call_gives_the_same_bits(cuda_lib, rows, cols):
    """With other memory, and with another stream's work beside it."""
    x, dy = values(rows, cols, BF16), values(rows, cols, BF16, seed=3)
    w, b = params(cols, F32)
    side = torch.cuda.Stream()

    def call():
        q, y, stats = cuda_lib.fp8_layernorm(x, w, b, with_y=True)
        g, _, _ = cuda_lib.fp8_layernorm(x, w, b, group=128)
        return (q.codes, q.scales(), y, stats, g.codes, g.scales()) + cuda_lib.layernorm_bwd(dy, x, w, stats)

    want = call()
    for i in range(10):
        torch.full((rows * cols + i,), float("nan"), device="cuda")
        with torch.cuda.stream(side):
            for _ in range(i % 3):
                torch.ones(rows, cols, device="cuda").mul_(2)
        assert all(torch.equal(p, q) for p, q in zip(call(), want))
    torch.cuda.synchronize()
