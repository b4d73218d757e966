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
