"""SwiGLU with 8-bit checkpoints on the GPU against the plain 64-bit reference.

The checkpoint holds BF16 inputs rounded to FP8: compared bit for bit.  What
passes through exp in FP32 is compared through tolerances: see `fuzz`."""
import numpy as np
import pytest
import torch

import lowbit_ref as ref
import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import workloads

pytestmark = pytest.mark.gpu
E4M3, E5M2 = ref.E4M3, ref.E5M2
FMTS = [pytest.param(E4M3, id="e4m3"), pytest.param(E5M2, id="e5m2")]


def gpu(bits):
    return workloads.from_bits(bits).cuda()


def data(rows, cols, seed, scale=1.5):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols)) * scale * np.exp(rng.normal(0, 0.7, (1, cols)))
    x[rng.random((rows, cols)) < 0.02] = 0.0
    return ref.f64_to_bf16_bits(x)


def fuzz(g):
    """Relative error of sigmoid(g) in FP32: exp(-g) through one product with
    log2(e) (half an ulp of |g| log2 e, that is |g| 2^-24 in the exponent), the
    fast power and the fast quotient (2 ulp each), 1 + exp and three products
    (half an ulp each): (|g| + 16) 2^-23 with room to spare."""
    return (np.abs(g) + 16) * 2.0 ** -22


TINY = 1e-36   # where exp(-g) leaves FP32's range the sigmoid is 0


def check_ckpt(q, x, fmt):
    """A stored half of the checkpoint: codes and scale bytes, bit for bit."""
    codes, scales = ref.fp8_quant(x, fmt)
    assert np.array_equal(q.scales().cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def check_fuzzy(codes, scales, v, tol, fmt):
    """Codes [rows, cols] and scale bytes in groups of 128 columns of a value
    known within tol: the scale is that of some amax in reach, and each code
    lies between the codes of v - tol and v + tol at that scale (the encoder is
    monotonic)."""
    lo = np.maximum(np.abs(v) - tol, 0)
    e_lo = ref.ue8m0(ref.groups(lo), fmt)
    e_hi = ref.ue8m0(ref.groups(np.abs(v) + tol), fmt)
    e = scales.astype(int) - 127
    assert ((e >= e_lo) & (e <= e_hi)).all(), np.argwhere(~((e >= e_lo) & (e <= e_hi)))[:4]
    s = np.exp2(np.repeat(e, 128, 1)[:, :v.shape[1]].astype(np.float64))
    t = ref.FP8[fmt]
    mag = codes & 0x7F
    assert (mag < len(t)).all()
    val = t[np.minimum(mag, len(t) - 1)] * np.where(codes & 0x80, -1.0, 1.0)

    def enc(x):
        return t[ref.nearest(t, np.abs(x) / s)] * np.sign(x)
    bad = ~((val >= enc(v - tol)) & (val <= enc(v + tol)))
    assert not bad.any(), (np.argwhere(bad)[:4], val[bad][:4], v[bad][:4])


SIZES = [(1, 1), (1, 8960), (2, 127), (3, 128), (5, 129), (37, 8960), (64, 1000), (130, 5001), (256, 384),
         (1, 18944), (9, 33000)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("fmt_h", FMTS)
def test_forward(cuda_lib, rows, cols, fmt, fmt_h):
    both = data(rows, 2 * cols, rows + cols)
    t = gpu(both)
    h, ck = fp8hg.fp8_swiglu_ckpt(t[:, :cols], t[:, cols:], fmt, fmt_h)
    x = ref.bf16_to_f64(both)
    g, u = x[:, :cols], x[:, cols:]
    check_ckpt(ck.gate, g, fmt)
    check_ckpt(ck.up, u, fmt)
    v = ref.swiglu(g, u)
    check_fuzzy(h.codes.cpu().numpy(), h.scales().cpu().numpy(), v, np.abs(v) * fuzz(g) + TINY, fmt_h)
    alone, none = fp8hg.fp8_swiglu_ckpt(t[:, :cols], t[:, cols:], fmt, fmt_h, checkpoint=False)
    assert none is None and torch.equal(alone.codes, h.codes) and torch.equal(alone.scales(), h.scales())


@pytest.mark.parametrize("shift", [0, 1, 8])
def test_forward_of_views(cuda_lib, shift):
    """gate and up as slices at any alignment; nothing beside the outputs changes."""
    rows, cols = 20, 300
    bits = data(rows, 2 * cols + 40, 3)
    t = gpu(bits)
    x = ref.bf16_to_f64(bits)
    g, u = slice(shift, shift + cols), slice(cols + 20 + shift, 2 * cols + 20 + shift)
    h, ck = fp8hg.fp8_swiglu_ckpt(t[:, g], t[:, u])
    check_ckpt(ck.gate, x[:, g], E4M3)
    check_ckpt(ck.up, x[:, u], E4M3)
    v = ref.swiglu(x[:, g], x[:, u])
    check_fuzzy(h.codes.cpu().numpy(), h.scales().cpu().numpy(), v, np.abs(v) * fuzz(x[:, g]) + TINY, E4M3)


def test_forward_writes_nothing_else(cuda_lib):
    """Outputs inside larger buffers, through the C entry."""
    from fp8_hybrid_granularity_gb300 import lowbit
    rows, cols, ld, lds = 5, 200, 256, 5
    t = gpu(data(rows, 2 * cols, 4))
    bufs = [torch.full((rows + 2, ld), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(3)]
    scs = [torch.full((rows + 2, lds), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(3)]
    p = [b[1:].data_ptr() for b in bufs]
    s = [b[1:].data_ptr() for b in scs]
    assert lowbit._fns().fp8_swiglu_ckpt(t.data_ptr(), t.data_ptr() + 2 * cols, rows, cols, 2 * cols, E4M3,
                                         p[0], ld, s[0], lds, E4M3, p[1], s[1], p[2], s[2], ld, lds, None) == 0
    torch.cuda.synchronize()
    for b, w in [(b, cols) for b in bufs] + [(b, 2) for b in scs]:
        assert (b[0] == 0xAB).all() and (b[-1] == 0xAB).all() and (b[:, w:] == 0xAB).all()


def test_forward_special_values(cuda_lib):
    """Groups of zeros, with NaN or an infinity, with large gates of both signs, with products past FP32."""
    rows, cols = 8, 384
    b = data(rows, 2 * cols, 6)
    b[0, :] = 0
    b[1, 5] = 0x7FC0                                       # gate: first group
    b[2, cols + 200] = 0xFF80                              # up: second group
    b[3, :cols] = ref.f64_to_bf16_bits(np.where(np.arange(cols) % 2, 300.0, -300.0))
    b[4, :] = 0x7F00                                       # 1.7e38: the product overflows
    t = gpu(b)
    h, ck = fp8hg.fp8_swiglu_ckpt(t[:, :cols], t[:, cols:])
    x = ref.bf16_to_f64(b)
    g, u = x[:, :cols], x[:, cols:]
    check_ckpt(ck.gate, g, E4M3)
    check_ckpt(ck.up, u, E4M3)
    hs, hc = h.scales().cpu().numpy(), h.codes.cpu().numpy()
    marked = np.zeros((rows, 3), bool)
    marked[1, 0] = marked[2, 1] = True
    marked[4, :] = True
    assert np.array_equal(hs == 0xFF, marked)
    assert (hc[np.repeat(marked, 128, 1)] == 0x7F).all()
    rest = [0, 3, 5, 6, 7]
    v = ref.swiglu(g[rest], u[rest])
    check_fuzzy(hc[rest], hs[rest], v, np.abs(v) * fuzz(g[rest]) + TINY, E4M3)


def checkpoint(rows, cols, fmt, seed, scale=1.5):
    """A stored checkpoint and its values."""
    vals, qs = [], []
    for i in range(2):
        codes, scales = ref.fp8_quant(ref.bf16_to_f64(data(rows, cols, seed + i, scale)), fmt)
        ld, ls = -(-cols // 16) * 16, -(-scales.shape[1] // 4) * 4
        c = torch.zeros(rows, ld, dtype=torch.uint8)
        c[:, :cols] = torch.from_numpy(codes)
        s = torch.zeros(rows, ls, dtype=torch.uint8)
        s[:, :scales.shape[1]] = torch.from_numpy(scales)
        qs.append(fp8hg.QTensor(c.cuda()[:, :cols], s.cuda(), fmt, fp8hg.GRAN_1x128, scales.shape[1]))
        vals.append(ref.fp8_values(codes, scales, fmt))
    return fp8hg.SwigluCkpt(*qs), vals[0], vals[1]


def grads_and_fuzz(g, u, dh):
    dg, du = ref.swiglu_grads(g, u, dh)
    s = ref.sigmoid(g)
    # dgate's factor s + g s (1 - s): both terms, and 1 - s near s = 1
    tg = np.abs(dh * u) * s * (1 + np.abs(g)) * fuzz(g) + np.abs(dh * u) * TINY + TINY
    tu = np.abs(du) * fuzz(g) + np.abs(dh) * TINY + TINY
    h = g * s * u
    return dg, du, h, tg, tu, np.abs(h) * fuzz(g) + TINY


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8960), (3, 127), (64, 129), (130, 5001), (256, 384), (2, 40000)])
@pytest.mark.parametrize("fmt", FMTS)
def test_backward(cuda_lib, rows, cols, fmt):
    ck, g, u = checkpoint(rows, cols, fmt, 10)
    bits = data(rows, cols, 12, 1e-3)
    dh = ref.bf16_to_f64(bits)
    dg, du, _, tg, tu, _ = grads_and_fuzz(g, u, dh)
    got = fp8hg.fp8_swiglu_ckpt_bwd(gpu(bits), ck).double().cpu().numpy()
    for d, t, p in ((dg, tg, got[:, :cols]), (du, tu, got[:, cols:])):
        err = np.abs(p - d)
        tol = t + 2.0 ** -8 * np.abs(d)
        assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])


def test_backward_views(cuda_lib):
    """dh unaligned, gradients into a slice of a wider buffer."""
    rows, cols = 12, 300
    ck, g, u = checkpoint(rows, cols, E4M3, 20)
    bits = data(rows, cols + 7, 22, 1e-3)
    want = fp8hg.fp8_swiglu_ckpt_bwd(gpu(bits)[:, 3:cols + 3].contiguous(), ck)
    wide = torch.full((rows, 2 * cols + 9), 3.0, dtype=torch.bfloat16, device="cuda")
    fp8hg.fp8_swiglu_ckpt_bwd(gpu(bits)[:, 3:cols + 3], ck, out=wide[:, 5:2 * cols + 5])
    assert torch.equal(wide[:, 5:2 * cols + 5], want)
    assert (wide[:, :5] == 3).all() and (wide[:, 2 * cols + 5:] == 3).all()


def test_backward_against_differences(cuda_lib):
    """The gradients against differences of the 64-bit forward at the checkpoint's values."""
    rows, cols = 16, 256
    ck, g, u = checkpoint(rows, cols, E4M3, 30)
    ones = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    got = fp8hg.fp8_swiglu_ckpt_bwd(ones, ck).double().cpu().numpy()
    eps = 1e-4
    ng = (ref.swiglu(g + eps, u) - ref.swiglu(g - eps, u)) / (2 * eps)
    nu = (ref.swiglu(g, u + eps) - ref.swiglu(g, u - eps)) / (2 * eps)
    # |f'''| <= 1 |u|: eps^2 |u| / 6, plus BF16's rounding and FP32's
    for n, p in ((ng, got[:, :cols]), (nu, got[:, cols:])):
        assert (np.abs(p - n) <= 2.0 ** -8 * np.abs(n) + 1e-6 * (1 + np.abs(u)) * (1 + np.abs(g))).all()


@pytest.mark.parametrize("rows,cols", [(128, 128), (256, 384), (384, 1536), (128, 2048)])
@pytest.mark.parametrize("fmt,fmt_t,fmt_h", [(E5M2, E5M2, E4M3), (E4M3, E5M2, E5M2), (E4M3, E4M3, E4M3)])
def test_backward_quantized(cuda_lib, rows, cols, fmt, fmt_t, fmt_h):
    ck, g, u = checkpoint(rows, cols, E4M3, 40)
    bits = data(rows, cols, 42, 1e-3)
    dg, du, h, tg, tu, th = grads_and_fuzz(g, u, ref.bf16_to_f64(bits))
    d, dt, ht = fp8hg.fp8_swiglu_ckpt_bwd_q(gpu(bits), ck, fmt, fmt_t, fmt_h)
    both, tol = np.concatenate([dg, du], 1), np.concatenate([tg, tu], 1)
    n = lambda q: (q.codes.cpu().numpy(), q.scales().cpu().numpy())
    check_fuzzy(*n(d), both, tol, fmt)
    check_fuzzy(*n(dt), both.T, tol.T, fmt_t)
    check_fuzzy(*n(ht), h.T, th.T, fmt_h)


def test_backward_special_values(cuda_lib):
    """A marked group of the checkpoint, NaN in dh, zeros, gates far out."""
    rows, cols = 128, 256
    ck, g, u = checkpoint(rows, cols, E4M3, 50)
    bits = data(rows, cols, 52, 1e-3)
    bits[5, 200] = 0x7FC0
    bits[9, :] = 0
    ck.gate.codes[3, :128] = 0x7F
    ck.gate.scale[3, 0] = 0xFF
    g[3, :128] = np.nan
    ck.gate.scale[7, 1] = 127 + 3                        # gates up to 448 * 8
    g[7, 128:] = ref.fp8_values(ck.gate.codes[7:8].cpu().numpy(), ck.gate.scales()[7:8].cpu().numpy(), E4M3)[0, 128:]
    dh = ref.bf16_to_f64(bits)
    dg, du, h, tg, tu, th = grads_and_fuzz(g, u, dh)
    got = fp8hg.fp8_swiglu_ckpt_bwd(gpu(bits), ck).double().cpu().numpy()
    d, dt, ht = fp8hg.fp8_swiglu_ckpt_bwd_q(gpu(bits), ck)
    both, tol = np.concatenate([dg, du], 1), np.concatenate([tg, tu], 1)
    assert np.array_equal(np.isnan(got), np.isnan(both))
    ok = ~np.isnan(both)
    assert (np.abs(got - both)[ok] <= (tol + 2.0 ** -8 * np.abs(both))[ok]).all()
    for q, v in ((d, both), (dt, both.T), (ht, h.T)):
        want = ref.groups(np.where(np.isnan(v), 1.0, 0.0)) > 0
        assert np.array_equal(q.scales().cpu().numpy() == 0xFF, want)
        assert (q.codes.cpu().numpy()[np.repeat(want, 128, 1)] == 0x7F).all()


def test_gradients_feed_the_fp8_products(cuda_lib):
    """The quantized gradients are operands of fp8_gemm_scaled as they are."""
    rows, cols, hid = 256, 256, 384
    ck, g, u = checkpoint(rows, cols, E4M3, 60)
    bits = data(rows, cols, 62, 1e-3)
    d, dt, ht = fp8hg.fp8_swiglu_ckpt_bwd_q(gpu(bits), ck, E5M2, E4M3, E4M3)
    x = torch.randn(rows, hid, device="cuda").bfloat16()
    w = torch.randn(2 * cols, hid, device="cuda").bfloat16()
    xt = fp8hg.fp8_quant_token(x, 128, E4M3, transpose=True)
    _, wt = fp8hg.fp8_quant_block128(w, E4M3, transposed_copy=True)
    val = lambda q: torch.from_numpy(ref.fp8_values(q.codes.cpu().numpy(), q.scales().cpu().numpy(), q.fmt)).cuda()
    dx = fp8hg.fp8_gemm_scaled(fp8hg.DGRAD, d, wt)
    dw = fp8hg.fp8_gemm_scaled(fp8hg.WGRAD, dt, xt, out_dtype=torch.float32)
    wv = ref.FP8[E4M3][wt.codes.cpu().numpy() & 0x7F] * np.where(wt.codes.cpu().numpy() & 0x80, -1, 1)
    wv = wv * np.exp2(np.repeat(np.repeat(wt.scales().cpu().numpy(), 128, 0), 128, 1).astype(float) - 127)
    for got, a, b in ((dx, val(d), torch.from_numpy(wv).cuda()), (dw, val(dt), val(xt))):
        c, s = a @ b.t(), a.abs() @ b.abs().t()
        assert ((got.double() - c).abs() <= 4e-3 * s + 2.0 ** -8 * c.abs() + 1e-30).all()


def test_empty_and_refusals(cuda_lib):
    z = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    h, ck = fp8hg.fp8_swiglu_ckpt(z[:, :128], z[:, 128:])
    assert h.codes.shape == (0, 128)
    assert fp8hg.fp8_swiglu_ckpt_bwd(z[:, :128].contiguous(), ck).shape == (0, 256)
    a = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    for g, u in ((a, a[:2]), (a.float(), a), (a, torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")[:, :128])):
        with pytest.raises(ValueError):
            fp8hg.fp8_swiglu_ckpt(g, u)
    _, ck = fp8hg.fp8_swiglu_ckpt(a, a)
    with pytest.raises(ValueError):
        fp8hg.fp8_swiglu_ckpt_bwd(a[:2], ck)
    with pytest.raises(fp8hg.Fp8hgError):
        fp8hg.fp8_swiglu_ckpt_bwd_q(a, ck)                # 4 rows


def test_on_another_stream_and_in_a_graph(cuda_lib):
    t = gpu(data(256, 768, 70))
    dh = gpu(data(256, 384, 71, 1e-3))
    h, ck = fp8hg.fp8_swiglu_ckpt(t[:, :384], t[:, 384:])
    want = fp8hg.fp8_swiglu_ckpt_bwd(dh, ck)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        h2, ck2 = fp8hg.fp8_swiglu_ckpt(t[:, :384], t[:, 384:])
        got = fp8hg.fp8_swiglu_ckpt_bwd(dh, ck2)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(h.codes, h2.codes)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(want)
    with torch.cuda.graph(g):
        _, ck3 = fp8hg.fp8_swiglu_ckpt(t[:, :384], t[:, 384:])
        fp8hg.fp8_swiglu_ckpt_bwd(dh, ck3, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("rows,cols", [(2048, 3840), (3968, 640), (128, 32768)])
def test_backward_quantized_over_many_tiles(cuda_lib, rows, cols):
    """More tiles than SMs, several per CTA: every stripe of 128 tokens comes out
    as it does alone (where no CTA has more than one tile to hand on)."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    rand = lambda: (torch.randn((rows, cols), generator=g, device="cuda") *
                    torch.exp(2 * torch.randn((rows, 1), generator=g, device="cuda"))).bfloat16()
    dh = rand()
    _, ck = fp8hg.fp8_swiglu_ckpt(rand(), rand())
    d, t, h = fp8hg.fp8_swiglu_ckpt_bwd_q(dh, ck)
    step = 128 if rows > 128 else 0
    for r in range(0, rows, 128):
        for c in range(0, cols, cols if step else 4096):
            n = cols if step else 4096
            part = fp8hg.SwigluCkpt(*(fp8hg.QTensor(q.codes[r:r + 128, c:c + n], q.scale[r:r + 128, c // 128:], q.fmt,
                                                    q.gran, n // 128) for q in (ck.gate, ck.up)))
            d1, t1, h1 = fp8hg.fp8_swiglu_ckpt_bwd_q(dh[r:r + 128, c:c + n], part)
            for half in (0, 1):
                at, to = half * cols + c, half * n
                assert torch.equal(d.codes[r:r + 128, at:at + n], d1.codes[:, to:to + n])
                assert torch.equal(d.scales()[r:r + 128, at // 128:(at + n) // 128],
                                   d1.scales()[:, to // 128:(to + n) // 128])
                assert torch.equal(t.codes[at:at + n, r:r + 128], t1.codes[to:to + n])
                assert torch.equal(t.scales()[at:at + n, r // 128:r // 128 + 1], t1.scales()[to:to + n])
            assert torch.equal(h.codes[c:c + n, r:r + 128], h1.codes)
            assert torch.equal(h.scales()[c:c + n, r // 128:r // 128 + 1], h1.scales())
    assert fp8hg.fp8hg_get_device_error() == 0
