"""Adapters where the arithmetic leaves one right answer: values of more bits than two
BF16 parts hold, and sums of values of one sign, where cut-off ends of sums add up."""
import pytest
import torch

import adapt_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# tokens, n, k, r, adapters: the results of few tokens in one kernel, rows as TMA takes
# them, odd ones, every padded rank, one chunk and several
SIZES = [(12, 132, 1032, 16, 2), (40, 264, 520, 64, 12), (300, 256, 520, 24, 3), (300, 1003, 517, 24, 3), (2500, 264, 4096, 64, 2),
         (700, 131, 2049, 128, 1), (700, 2049, 131, 128, 2), (1500, 200, 72, 16, 1)]


def three_parts(gen, rows, long_side, g, r):
    """x [rows, long_side] and w [g, r, long_side] whose products have 22 bits: x is 1 or -1
    in three columns, and w is there a whole number of 2^-7, one of 2^-15 and one of
    2^-21, each of one BF16: x w^T is a whole number of 2^-21 below 2, one and the same in
    every order of its additions, exact in FP32 and where a product is cut at 2^-23 of
    the largest one.  Its two first BF16 parts have steps of 2^-7 and mostly 2^-16 or
    2^-17; an odd number of 2^-21 is left for the third.  Elsewhere x is 0 and w anything."""
    x = torch.zeros(rows, long_side)
    w = torch.randn(g, r, long_side, generator=gen)
    for col, lo, hi, odd, step in ((3, 128, 240, 0, -7), (long_side // 2, 1, 255, 0, -15), (long_side - 1, 16, 31, 1, -21)):
        x[:, col] = torch.randint(0, 2, (rows,), generator=gen) * 2.0 - 1
        w[:, :, col] = (torch.randint(lo, hi + 1, (g, r), generator=gen) * (1 + odd) + odd) * 2.0 ** step
    return x.bfloat16().cuda(), w.bfloat16().cuda()


def one_of_each(gen, g, r, n):
    """w [g, r, n] with one value a column, a power of two or its negative."""
    w = torch.zeros(g, r, n)
    at = torch.randint(0, r, (g, n), generator=gen)
    w.scatter_(1, at.unsqueeze(1), (torch.exp2(torch.randint(-3, 4, (g, n), generator=gen).float()) *
                                    (torch.randint(0, 2, (g, n), generator=gen) * 2.0 - 1)).unsqueeze(1))
    return w.bfloat16().cuda()


def ids_of(gen, t, g):
    return torch.randint(-1 if g > 1 else 0, g, (t,), generator=gen, dtype=torch.int32).cuda()


def spread(ids, g, cols):
    """[tokens, cols]: in every column one token of each adapter has a 1."""
    x = torch.zeros(ids.shape[0], cols, device="cuda")
    for i in range(g):
        rows = (ids == i).nonzero().squeeze(1)
        if len(rows):
            x[rows[torch.arange(cols, device="cuda") % len(rows)], torch.arange(cols, device="cuda")] = 1.0
    return x.bfloat16()


@pytest.mark.parametrize("size", SIZES)
def test_results_have_all_bits(cuda_lib, size):
    """v, y in FP32 and its rounding to BF16."""
    t, n, k, r, g = size
    gen = torch.Generator().manual_seed(t + n)
    x, a = three_parts(gen, t, k, g, r)
    b = one_of_each(gen, g, r, n).transpose(1, 2).contiguous()
    ids, scale = ids_of(gen, t, g), torch.exp2(torch.arange(g, device="cuda") % 5 - 2.0)
    want_v, _, want, _ = ref.lora(x, a, b, scale, None, ids)
    plan = cuda_lib.lora_plan(ids, g)
    w = cuda_lib.LoraAdapters(a, b, scale)
    y, v = cuda_lib.lora_add(None, x, w, plan, keep=True, out_dtype=F32)
    assert torch.equal(v.double(), want_v)
    assert torch.equal(y.double(), want)
    y, _ = cuda_lib.lora_add(torch.zeros(t, n, dtype=F32, device="cuda"), x, w, plan)
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("size", SIZES)
def test_gradients_have_all_bits(cuda_lib, size):
    """dx and dA from dv, dB from v of 24 bits, in FP32."""
    t, n, k, r, g = size
    gen = torch.Generator().manual_seed(t + k)
    dy, b = three_parts(gen, t, n, g, r)
    b = b.transpose(1, 2).contiguous()
    a = one_of_each(gen, g, r, k)
    ids, scale = ids_of(gen, t, g), torch.exp2(torch.arange(g, device="cuda") % 5 - 2.0)
    x, v = spread(ids, g, k), torch.randn(t, r, generator=gen).cuda()
    plan = cuda_lib.lora_plan(ids, g)
    w = cuda_lib.LoraAdapters(a, b, scale)
    (wx, _), (wa, _), _ = ref.lora_bwd(dy, x, v.double(), a, b, scale, None, ids)
    dx, da, _ = cuda_lib.lora_add_bwd(dy, x, v, w, plan, out_dtype=F32)
    assert torch.equal(dx.double(), wx) and torch.equal(da.double(), wa)
    only, _, _ = cuda_lib.lora_add_bwd(dy, None, None, w, plan, out_dtype=F32, params=False)
    assert torch.equal(only, dx)
    dy = spread(ids, g, n)
    _, _, (wb, _) = ref.lora_bwd(dy, x, v.double(), a, b, scale, None, ids)
    _, _, db = cuda_lib.lora_add_bwd(dy, x, v, w, plan)
    assert torch.equal(db.double(), wb)


def lean(got, want):
    return abs(float(((got.double() - want) / want).mean()))


# A sum of 16 products is cut off at the running sum's last bit, 2^-23 of it or less: half
# of that is lost on the average.  After m such sums, the running one growing evenly,
# that is (m + 1) / 2 * 2^-24 of the result.  What is added in registers is rounded,
# as often up as down.
LEAN_48, LEAN_32 = 24.5 * 2.0 ** -24, 16.5 * 2.0 ** -24


@pytest.mark.parametrize("t,k,r", [(19500, 20000, 16), (19500, 9000, 128), (300, 20000, 32), (9, 49152, 16), (20, 100000, 128)])
def test_sums_over_a_long_side_do_not_lean(cuda_lib, t, k, r):
    """x A^T of values of one sign: at most 48 sums of 16 behind one another, however long
    the side and however few CTAs there are for it."""
    g = torch.Generator(device="cuda").manual_seed(t)
    x = torch.randn(t, k, generator=g, device="cuda").abs_().bfloat16()
    a, b = torch.randn(1, r, k, generator=g, device="cuda").abs().bfloat16(), torch.ones(1, 64, r, dtype=BF16, device="cuda")
    plan = cuda_lib.lora_plan(torch.zeros(t, dtype=torch.int32, device="cuda"), 1)
    _, v = cuda_lib.lora_add(None, x, cuda_lib.LoraAdapters(a, b), plan, keep=True)
    rows = torch.arange(0, t, max(1, t // 100), device="cuda")
    assert lean(v[rows], x[rows].double() @ a[0].double().t()) < LEAN_48


@pytest.mark.parametrize("t,r", [(8192, 16), (20000, 128), (5000, 64)])
def test_sums_over_the_tokens_do_not_lean(cuda_lib, t, r):
    """dB of values of one sign: at most 32 sums of 16 behind one another."""
    g = torch.Generator(device="cuda").manual_seed(t)
    f = lambda *s: torch.randn(*s, generator=g, device="cuda").abs_()  # noqa: E731
    dy, x, v = f(t, 1000).bfloat16(), f(t, 64).bfloat16(), f(t, r)
    w = cuda_lib.LoraAdapters(f(1, r, 64).bfloat16(), f(1, 1000, r).bfloat16())
    plan = cuda_lib.lora_plan(torch.zeros(t, dtype=torch.int32, device="cuda"), 1)
    _, _, db = cuda_lib.lora_add_bwd(dy, x, v, w, plan)
    assert lean(db[0, :200], dy[:, :200].double().t() @ v.double()) < LEAN_32
