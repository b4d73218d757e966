"""A SwiGLU MLP on 4-bit weights, its training step and its decoding step.

    python examples/mlp_4bit.py [--tokens 8192] [--hidden 1536] [--mlp 8960] [--kind nv]

  forward    gate | up = x W_gu^T        4-bit product, x quantized in the call
             h = silu(gate) * up         one pass: FP8 h, FP8 checkpoints of gate and up
             y = h W_down^T              FP8 product
  backward   dh = dy W_down              FP8 product
    fp8      dgate, dup, h^T             one pass over dh and the checkpoints, both directions
             dx = [dgate dup] W_gu       FP8 products (dgate, dup and x transposed per 128 tokens)
             dW_gu = [dgate dup]^T x
    fp4      the gradients in BF16, quantized to 4 bits along both directions
             from one read; dx and dW_gu as 4-bit products
  decoding   a few tokens: the 4-bit product quantizes its rows itself, SwiGLU
             keeps no checkpoint, and the whole step is one CUDA graph

Between the calls there are only device tensors; nothing is read back.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import fp8_hybrid_granularity_gb300 as fp8hg


class Mlp:
    """Weights [2 mlp, hidden] (gate above up) and [hidden, mlp], BF16."""

    def __init__(self, w_gu, w_down, kind=None):
        self.kind = fp8hg.FP4_NV if kind is None else kind
        self.mlp = w_down.shape[1]
        ts = fp8hg.fp4_tensor_scale(w_gu) if self.kind == fp8hg.FP4_NV else None
        # 4 bits along both of its axes: forward and data gradient
        self.gu, self.gu_t = fp8hg.fp4_quant_dual(w_gu, self.kind, ts)
        # FP8: the data gradient of gate | up, and the down projection
        _, self.gu8_t = fp8hg.fp8_quant_block128(w_gu, transposed_copy=True)
        self.down, self.down_t = fp8hg.fp8_quant_block128(w_down, transposed_copy=True)

    def _scale(self, x):
        return fp8hg.fp4_tensor_scale(x) if self.kind == fp8hg.FP4_NV else None

    def forward(self, x, checkpoint=True):
        """y, and what backward needs."""
        gu = fp8hg.fp4_linear(x, self.gu, self._scale(x))
        h, ckpt = fp8hg.fp8_swiglu_ckpt(gu[:, :self.mlp], gu[:, self.mlp:], checkpoint=checkpoint)
        return fp8hg.fp8_gemm_scaled(fp8hg.FPROP, h, self.down), ckpt

    def backward(self, x, ckpt, dy):
        """dx, dW_gu, dW_down with the products of gate | up in FP8."""
        dy_q, dy_t = fp8hg.fp8_quant_token_dual(dy)
        dh = fp8hg.fp8_gemm_scaled(fp8hg.DGRAD, dy_q, self.down_t)
        d, d_t, h_t = fp8hg.fp8_swiglu_ckpt_bwd_q(dh, ckpt)
        x_t = fp8hg.fp8_quant_token(x, 128, transpose=True)
        dx = fp8hg.fp8_gemm_scaled(fp8hg.DGRAD, d, self.gu8_t)
        dw_gu = fp8hg.fp8_gemm_scaled(fp8hg.WGRAD, d_t, x_t, out_dtype=torch.float32)
        dw_down = fp8hg.fp8_gemm_scaled(fp8hg.WGRAD, dy_t, h_t, out_dtype=torch.float32)
        return dx, dw_gu, dw_down

    def backward_fp4(self, x, ckpt, dy):
        """dx and dW_gu with 4-bit products."""
        dh = fp8hg.fp8_gemm_scaled(fp8hg.DGRAD, fp8hg.fp8_quant_token(dy), self.down_t)
        d = fp8hg.fp8_swiglu_ckpt_bwd(dh, ckpt)
        d4, d4_t = fp8hg.fp4_quant_dual(d, self.kind, self._scale(d))
        x4_t = fp8hg.fp4_quant(x, self.kind, self._scale(x), transpose=True)
        dx = fp8hg.fp4_gemm_scaled(d4, self.gu_t)
        dw_gu = fp8hg.fp4_gemm_scaled(d4_t, x4_t, out_dtype=torch.float32)
        return dx, dw_gu

    def decode(self, x, gu):
        """y for a few tokens.  gu [128 n, 2 mlp]: a buffer whose rows past the
        tokens hold zeros, because the FP8 product takes whole blocks of 128 rows."""
        fp8hg.fp4_linear(x, self.gu, self._scale(x), out=gu[:x.shape[0]])
        h, _ = fp8hg.fp8_swiglu_ckpt(gu[:, :self.mlp], gu[:, self.mlp:], checkpoint=False)
        return fp8hg.fp8_gemm_scaled(fp8hg.FPROP, h, self.down)[:x.shape[0]]

    def decoder(self, tokens):
        """x [tokens, hidden], y [tokens, hidden] and a graph that computes y from x."""
        x = torch.zeros((tokens, self.gu.k), dtype=torch.bfloat16, device="cuda")
        gu = torch.zeros(((tokens + 127) // 128 * 128, 2 * self.mlp), dtype=torch.bfloat16, device="cuda")
        self.decode(x, gu)                   # one-time set-up outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = self.decode(x, gu)
        return x, y, graph


def reference(x, w_gu, w_down, dy):
    """y, dx, dW_gu, dW_down in FP32 on unquantized tensors."""
    x, w_gu, w_down, dy = (t.float() for t in (x, w_gu, w_down, dy))
    g, u = (x @ w_gu.T).chunk(2, dim=1)
    s = torch.sigmoid(g)
    h = g * s * u
    dh = dy @ w_down
    d = torch.cat((dh * u * s * (1 + g * (1 - s)), dh * g * s), dim=1)
    return h @ w_down.T, d @ w_gu, d.T @ x, dy.T @ h


def relative(a, b):
    return float((a.float() - b).norm() / b.norm())


def timed(fn, n=20):
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(n):
        fn()
    t1.record()
    torch.cuda.synchronize()
    return t0.elapsed_time(t1) / n * 1e3


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=8192)
    p.add_argument("--hidden", type=int, default=1536)
    p.add_argument("--mlp", type=int, default=8960)
    p.add_argument("--kind", choices=("mx", "nv"), default="nv")
    a = p.parse_args()
    if a.tokens % 128 or a.hidden % 128 or a.mlp % 128:
        p.error("tokens, hidden and mlp must be multiples of 128 (the FP8 backward products)")
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda r, c, s: (torch.randn((r, c), generator=gen, device="cuda") * s).bfloat16()
    x, dy = rand(a.tokens, a.hidden, 1.0), rand(a.tokens, a.hidden, 1.0)
    w_gu, w_down = rand(2 * a.mlp, a.hidden, a.hidden ** -0.5), rand(a.hidden, a.mlp, a.mlp ** -0.5)
    m = Mlp(w_gu, w_down, fp8hg.FP4_NV if a.kind == "nv" else fp8hg.FP4_MX)

    y, ckpt = m.forward(x)
    got8, got4 = m.backward(x, ckpt, dy), m.backward_fp4(x, ckpt, dy)
    ry, rdx, rdw, rdd = reference(x, w_gu, w_down, dy)
    print("relative to FP32: y %.3f | FP8 backward dx %.3f dW_gu %.3f dW_down %.3f | 4-bit backward dx %.3f dW_gu %.3f" %
          (relative(y, ry), relative(got8[0], rdx), relative(got8[1], rdw), relative(got8[2], rdd),
           relative(got4[0], rdx), relative(got4[1], rdw)))
    print("training, %d tokens: forward %.0f us, FP8 backward %.0f us, 4-bit backward (without dW_down) %.0f us" %
          (a.tokens, timed(lambda: m.forward(x)), timed(lambda: m.backward(x, ckpt, dy)),
           timed(lambda: m.backward_fp4(x, ckpt, dy))))
    for n in (1, 4, 32):
        xs, ys, graph = m.decoder(n)
        xs.copy_(x[:n])
        graph.replay()
        print("decoding %2d tokens: %.1f us a step, y as in the forward pass to %.1e" %
              (n, timed(graph.replay, 100), relative(ys, y[:n].float())))


if __name__ == "__main__":
    main()
