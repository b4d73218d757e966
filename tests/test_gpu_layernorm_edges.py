"""Layer norm at the edges of what a call may be given: rows whose sums are exact, so
that mean and rstd have one right value."""
import pytest
import torch

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
