"""Fine-tuning and serving beside a frozen 4-bit projection: the norm before it and
low-rank adapters next to it, which are all that is trained.

    python examples/adapters_4bit.py [--tokens 4096] [--hidden 1536] [--out 8960] [--rank 16] [--adapters 4] [--kind nv]

  forward    h = layer norm of x               BF16, mean and rstd kept
             y = h W^T                         4-bit product, h quantized in the call
             y += s_g (h A_g^T) B_g^T          each token's own adapter; h A^T kept
  backward   dh = dy W                         4-bit product, dy quantized
             dh += s_g dy B_g A_g, dA, dB      one call
             dx = residual's gradient + d(norm), dw, db
  decoding   a few tokens of different adapters, the whole step one CUDA graph

Between the calls there are only device tensors; nothing is read back.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import fp8_hybrid_granularity_gb300 as fp8hg


class AdaptedProjection:
    """W [out, hidden] in 4 bits, frozen; the norm's weight and bias and the adapters
    A [adapters, rank, hidden], B [adapters, out, rank] are trained."""

    def __init__(self, w, norm_weight, norm_bias, a, b, scale=None, ranks=None, kind=None):
        self.kind = fp8hg.FP4_NV if kind is None else kind
        ts = fp8hg.fp4_tensor_scale(w) if self.kind == fp8hg.FP4_NV else None
        # along both of its axes: forward and data gradient
        self.w, self.w_t = fp8hg.fp4_quant_dual(w, self.kind, ts)
        self.norm_weight, self.norm_bias = norm_weight, norm_bias
        self.adapters = fp8hg.LoraAdapters(a, b, scale, ranks)

    def _scale(self, x):
        return fp8hg.fp4_tensor_scale(x) if self.kind == fp8hg.FP4_NV else None

    def forward(self, x, plan, keep=True):
        """y, and what backward needs."""
        h, stats = fp8hg.layernorm(x, self.norm_weight, self.norm_bias, out_dtype=torch.bfloat16)
        y = fp8hg.fp4_linear(h, self.w, self._scale(h))
        y, v = fp8hg.lora_add(y, h, self.adapters, plan, out=y, keep=keep)
        return y, (h, stats, v)

    def backward(self, x, plan, kept, dy, d_residual=None):
        """dx (with the gradient of the residual that bypasses the block), and the
        gradients of the norm's weight and bias and of A and B, in FP32."""
        h, stats, v = kept
        dh = fp8hg.fp4_gemm_scaled(fp8hg.fp4_quant(dy, self.kind, self._scale(dy)), self.w_t)
        dh, da, db = fp8hg.lora_add_bwd(dy, h, v, self.adapters, plan, base=dh, out=dh)
        dx, dw, dbias = fp8hg.layernorm_bwd(dh, x, self.norm_weight, stats, add=d_residual)
        return dx, dw, dbias, da, db


def block(hidden, out, rank, adapters, kind=None, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return AdaptedProjection((0.02 * r(out, hidden)).bfloat16(), 1 + 0.1 * r(hidden), 0.1 * r(hidden),
                             (r(adapters, rank, hidden) / hidden ** 0.5).bfloat16(), (0.05 * r(adapters, out, rank)).bfloat16(),
                             torch.full((adapters,), 2.0, device="cuda"), kind=kind)


def timed(step, reps=20):
    for _ in range(3):
        step()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        step()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / reps


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 1536), ("out", 8960), ("rank", 16), ("adapters", 4)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--kind", choices=["mx", "nv"], default="nv")
    o = p.parse_args()
    b = block(o.hidden, o.out, o.rank, o.adapters, {"mx": fp8hg.FP4_MX, "nv": fp8hg.FP4_NV}[o.kind])
    x = torch.randn(o.tokens, o.hidden, device="cuda")
    dy = (1e-3 * torch.randn(o.tokens, o.out, device="cuda")).bfloat16()
    # requests of 128 tokens, one adapter each
    plan = fp8hg.lora_plan((torch.arange(o.tokens, device="cuda") // 128 % o.adapters).int(), o.adapters)

    def step():
        y, kept = b.forward(x, plan)
        return b.backward(x, plan, kept, dy, d_residual=x)
    print(f"training step, {o.tokens} tokens: {timed(step):.3f} ms")

    few = x[:8].contiguous()
    plan8 = fp8hg.lora_plan((torch.arange(8, device="cuda") % o.adapters).int(), o.adapters)
    b.forward(few, plan8, keep=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(few, plan8, keep=False)
    print(f"decoding step, 8 tokens: {timed(graph.replay) * 1e3:.1f} us")
    if fp8hg.fp8hg_get_device_error() != 0:
        raise SystemExit("device error")


if __name__ == "__main__":
    main()
