"""The 4-bit and SwiGLU calls at the edges of what they accept: streams given by
handle, operands of one row, scales far apart, very long rows, limits that run
out late in a product."""
import numpy as np
import pytest
import torch

import lowbit_ref as ref
import fp8_hybrid_granularity_gb300 as fp8hg

pytestmark = pytest.mark.gpu
MX, NV = ref.MX, ref.NV
KINDS = [pytest.param(MX, id="mx"), pytest.param(NV, id="nv")]


def rand(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((rows, cols), generator=g, device="cuda").bfloat16()


def test_handle_0_is_the_default_stream(cuda_lib):
    """A call given the default stream by its handle runs after what that stream
    still has to do, whichever stream is current."""
    assert torch.cuda.default_stream().cuda_stream == 0
    src = rand(512, 2048, 1)
    want = fp8hg.fp4_quant(src, MX)
    side = torch.cuda.Stream()
    for _ in range(3):
        x = torch.zeros_like(src)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        x.copy_(src)
        with torch.cuda.stream(side):
            got = fp8hg.fp4_quant(x, MX, stream=0)
        torch.cuda.synchronize()
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scale, want.scale)


def one_row(x, stride):
    """The values of x [1, n] in a row whose stride says nothing."""
    out = torch.empty(4 * (x.shape[1] + stride), dtype=x.dtype, device=x.device).as_strided(x.shape, (stride, 1))
    return out.copy_(x)


@pytest.mark.parametrize("stride", [1, 301, 5000])
@pytest.mark.parametrize("n", [257, 304])
def test_strides_of_one_row(cuda_lib, n, stride):
    """One row gives the same with any row stride, in each operand of each call."""
    x, up, dh = rand(1, n, 2), rand(1, n, 3), rand(1, n, 4)
    odd = one_row(x, stride)
    h, ck = fp8hg.fp8_swiglu_ckpt(x, up)
    for g, u in ((odd, up), (x, one_row(up, stride))):
        h2, ck2 = fp8hg.fp8_swiglu_ckpt(g, u)
        for a, b in ((h, h2), (ck.gate, ck2.gate), (ck.up, ck2.up)):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales(), b.scales())
    want = fp8hg.fp8_swiglu_ckpt_bwd(dh, ck)
    ck2.gate.codes = one_row(ck.gate.codes, stride)
    ck2.up.scale = one_row(ck.up.scale, stride)
    assert torch.equal(fp8hg.fp8_swiglu_ckpt_bwd(one_row(dh, stride), ck2), want)
    for kind in (MX, NV):
        w = fp8hg.fp4_quant(rand(40, n, 5), kind)
        q = fp8hg.fp4_quant(x, kind)
        q2 = fp8hg.fp4_quant(odd, kind)
        assert torch.equal(q.scales(), q2.scales())
        y, v = fp8hg.fp4_gemm_scaled(q, w), fp8hg.fp4_dequant(q)
        q2.codes = one_row(q.codes, stride)
        assert torch.equal(fp8hg.fp4_gemm_scaled(q2, w), y) and torch.equal(fp8hg.fp4_dequant(q2), v)
        assert torch.equal(fp8hg.fp4_linear(odd, w), y)
        for out in (torch.bfloat16, torch.float32):
            to = one_row(y.to(out), stride)
            fp8hg.fp4_gemm_scaled(q, w, out=to)
            assert torch.equal(to, fp8hg.fp4_gemm_scaled(q, w, out_dtype=out))
