"""Norm, frozen 4-bit projection and adapters as they are used together
(examples/adapters_4bit.py), the training step and the captured decoding step."""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

import adapt_ref as ref

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "adapters_4bit.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("adapters_4bit", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def batch(t, hidden, out, adapters, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(t, hidden, generator=g, device="cuda")
    dy = (0.1 * torch.randn(t, out, generator=g, device="cuda")).bfloat16()
    ids = (torch.arange(t, device="cuda") // 50 % (adapters + 1) - 1).int()       # every so often no adapter
    return x, dy, ids


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("t,hidden,out,rank", [(1, 256, 512, 16), (300, 384, 520, 24), (1000, 1536, 1000, 64)])
def test_training_step(cuda_lib, example, kind, t, hidden, out, rank):
    b = example.block(hidden, out, rank, 3, kind)
    x, dy, ids = batch(t, hidden, out, 3)
    plan = cuda_lib.lora_plan(ids, 3)
    y, (h, stats, v) = b.forward(x, plan)
    dx, dw, dbias, da, db = b.backward(x, plan, (h, stats, v), dy, d_residual=x)
    ad = b.adapters

    # each stage against 64 bits on what the stage before it gave
    mean, rstd, want, tol = ref.norm(x, b.norm_weight, b.norm_bias, 1e-5)
    ref.close(h, want, tol + ref.half_step(h.dtype) * 1.01 * want.abs(), "h")
    base = cuda_lib.fp4_linear(h, b.w, b._scale(h))
    want_v, vmag, add, mag = ref.lora(h, ad.a, ad.b, ad.scale, None, ids)
    want = base.double() + add
    ref.close(y, want, ref.MMA * mag + ref.half_step(y.dtype) * 1.01 * want.abs(), "y")
    ref.close(v, want_v, ref.MMA * vmag, "v")
    dh0 = cuda_lib.fp4_gemm_scaled(cuda_lib.fp4_quant(dy, b.kind, b._scale(dy)), b.w_t)
    (gx, mx), (ga, ma), (gb, mb) = ref.lora_bwd(dy, h, v, ad.a, ad.b, ad.scale, None, ids)
    ref.close(da, ga, ref.MMA * ma + ref.U * ga.abs(), "dA")
    ref.close(db, gb, ref.MMA * mb + ref.U * gb.abs(), "dB")
    dh = cuda_lib.lora_add_bwd(dy, h, v, ad, plan, base=dh0)[0]
    want = dh0.double() + gx
    ref.close(dh, want, ref.MMA * mx + ref.half_step(dh.dtype) * 1.01 * want.abs(), "dh")
    for got, (want, tol), what in zip((dx, dw, dbias), ref.norm_bwd(dh, x, b.norm_weight, stats, x), ("dx", "dw", "db")):
        ref.close(got, want, tol + ref.U * want.abs() + 1e-37, what)
    assert cuda_lib.fp8hg_get_device_error() == 0


def test_two_captured_steps(cuda_lib, example):
    """Decoding steps of two graphs that replay in turn, with other calls between."""
    b = example.block(256, 512, 16, 3)
    out, graphs, inputs = [], [], []
    for i in range(2):
        x, _, ids = batch(4 + i, 256, 512, 3, seed=i)
        ids = (torch.arange(4 + i, device="cuda") % 3).int()
        plan = cuda_lib.lora_plan(ids, 3)
        b.forward(x, plan, keep=False)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, _ = b.forward(x, plan, keep=False)
        out.append(y), graphs.append(g), inputs.append((x, plan))
    for rep in range(3):
        for x, _ in inputs:
            x.normal_()
        for g in graphs:
            g.replay()
        want = [b.forward(x, plan, keep=False)[0] for x, plan in inputs]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), rep


def test_command(cuda_lib):
    r = subprocess.run([sys.executable, PATH, "--tokens", "700", "--hidden", "256", "--out", "512", "--kind", "mx"], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "training step" in r.stdout and "decoding step" in r.stdout
