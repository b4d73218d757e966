"""The 4-bit MLP example: its steps against the same steps in 64 bits."""
import os
import sys

import numpy as np
import pytest
import torch

import fp8_hybrid_granularity_gb300 as fp8hg

sys.path.insert(0, os.path.join(os.path.dirname(__file__), "..", "examples"))
import mlp_4bit

pytestmark = pytest.mark.gpu


def q64(q):
    """Values of an FP8 operand with 1x128 scales, or of a 4-bit one, in 64 bits."""
    if isinstance(q, fp8hg.Fp4Tensor):
        return fp8hg.fp4_dequant(q, out_dtype=torch.float32).double()
    dt = torch.float8_e4m3fn if q.fmt == fp8hg.E4M3 else torch.float8_e5m2
    s = torch.ldexp(torch.ones((), device="cuda", dtype=torch.float64), q.scales().int() - 127)
    n = -(-q.codes.shape[1] // s.shape[1])
    return q.codes.view(dt).double() * s.repeat_interleave(n, dim=1)[:, :q.codes.shape[1]]


def bound(a, b, k, bf16=True):
    """|a| |b|^T and the product: FP32 accumulation (k + 16 roundings at most)
    and one rounding to BF16."""
    ref, mag = a @ b.T, a.abs() @ b.abs().T
    return ref, mag * (k + 16) * 2.0 ** -24 + (ref.abs() * 2.0 ** -8 if bf16 else 0) + 1e-30


@pytest.mark.parametrize("kind", ("mx", "nv"))
@pytest.mark.parametrize("tokens,hidden,mlp", ((128, 256, 384), (384, 384, 640)))
def test_training_step(cuda_lib, kind, tokens, hidden, mlp):
    gen = torch.Generator(device="cuda").manual_seed(tokens + hidden)
    rand = lambda r, c, s: (torch.randn((r, c), generator=gen, device="cuda") * s).bfloat16()
    x, dy = rand(tokens, hidden, 1.0), rand(tokens, hidden, 0.5)
    w_gu, w_down = rand(2 * mlp, hidden, hidden ** -0.5), rand(hidden, mlp, mlp ** -0.5)
    m = mlp_4bit.Mlp(w_gu, w_down, fp8hg.FP4_NV if kind == "nv" else fp8hg.FP4_MX)
    y, ckpt = m.forward(x)
    dx, dw_gu, dw_down = m.backward(x, ckpt, dy)
    dx4, dw4 = m.backward_fp4(x, ckpt, dy)

    # forward: the 4-bit product, then SwiGLU of it (BF16) to FP8, one rounding
    # of 2^-4 and the fast exponential (2^-19) apart, with a step below the
    # smallest normal of the group's scale
    x4 = q64(fp8hg.fp4_quant(x, m.kind, m._scale(x)))
    ref, tol = bound(x4, q64(m.gu), hidden)
    gu = fp8hg.fp4_linear(x, m.gu, m._scale(x))
    assert ((gu.double() - ref).abs() <= tol).all()
    g, u = gu.double().chunk(2, dim=1)
    h, ck = fp8hg.fp8_swiglu_ckpt(gu[:, :mlp], gu[:, mlp:])
    assert torch.equal(ck.gate.codes, ckpt.gate.codes) and torch.equal(ck.up.codes, ckpt.up.codes)
    s = torch.sigmoid(g)
    ulp = lambda q, n: torch.ldexp(torch.ones((), device="cuda", dtype=torch.float64),
                                   q.scales().int() - 127).repeat_interleave(n, dim=1)
    want = g * s * u
    assert ((q64(h) - want).abs() <= want.abs() * (2.0 ** -4 + 2.0 ** -18) + ulp(h, 128) * 2.0 ** -9).all()

    # backward from the checkpoint's values
    g, u = q64(ckpt.gate), q64(ckpt.up)
    s = torch.sigmoid(g)
    dh = fp8hg.fp8_gemm_scaled(fp8hg.DGRAD, fp8hg.fp8_quant_token(dy), m.down_t)
    d64 = torch.cat((dh.double() * u * s * (1 + g * (1 - s)), dh.double() * g * s), dim=1)
    d, d_t, h_t = fp8hg.fp8_swiglu_ckpt_bwd_q(dh, ckpt)
    # 1 + g (1 - s) cancels near g = -1.28: 2^-18 of its terms
    terms = torch.cat((dh.double().abs() * u.abs() * s * (1 + g.abs()), (dh.double() * g * s).abs()), dim=1)
    assert ((q64(d) - d64).abs() <= d64.abs() * 2.0 ** -3 + terms * 2.0 ** -18 + ulp(d, 128) * 2.0 ** -16).all()
    ref, tol = bound(q64(d_t), q64(fp8hg.fp8_quant_token(x, 128, transpose=True)), tokens, bf16=False)
    assert ((dw_gu.double() - ref).abs() <= tol).all()
    _, dy_t = fp8hg.fp8_quant_token_dual(dy)
    ref, tol = bound(q64(dy_t), q64(h_t), tokens, bf16=False)
    assert ((dw_down.double() - ref).abs() <= tol).all()
    assert dx.shape == x.shape

    # 4-bit backward: the BF16 gradients, quantized both ways
    db = fp8hg.fp8_swiglu_ckpt_bwd(dh, ckpt)
    a, a_t = fp8hg.fp4_quant_dual(db, m.kind, m._scale(db))
    ref, tol = bound(q64(a), q64(m.gu_t), 2 * mlp)
    assert ((dx4.double() - ref).abs() <= tol).all()
    xt = fp8hg.fp4_quant(x, m.kind, m._scale(x), transpose=True)
    ref, tol = bound(q64(a_t), q64(xt), tokens, bf16=False)
    assert ((dw4.double() - ref).abs() <= tol).all()

    # all of it near the unquantized step: an E2M1 element is off by at most a
    # quarter of itself or of a scale unit (a third of the block's maximum
    # rounded to a power of two at worst), E4M3 and E5M2 by 2^-4 and 2^-3;
    # products of two such operands, and SwiGLU's slope, stay below one half
    for got, want in zip((y, dx, dw_gu, dw_down, dx4, dw4),
                         (lambda r: (r[0], r[1], r[2], r[3], r[1], r[2]))(mlp_4bit.reference(x, w_gu, w_down, dy))):
        assert mlp_4bit.relative(got, want) < 0.5


@pytest.mark.parametrize("tokens", (1, 4, 5))
def test_decoding_step(cuda_lib, tokens):
    """The graph's replay gives what the calls give, for new inputs too."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    rand = lambda r, c, s: (torch.randn((r, c), generator=gen, device="cuda") * s).bfloat16()
    m = mlp_4bit.Mlp(rand(768, 256, 0.06), rand(256, 384, 0.05))
    gu = torch.zeros((128, 768), dtype=torch.bfloat16, device="cuda")
    xs, ys, graph = m.decoder(tokens)
    for _ in range(2):
        x = rand(tokens, 256, 1.0)
        xs.copy_(x)
        graph.replay()
        want = m.decode(x, gu)
        torch.cuda.synchronize()
        assert torch.equal(ys, want) and bool(torch.isfinite(ys.float()).all())
