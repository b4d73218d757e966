"""4-bit quantization and products on the GPU against the plain 64-bit
references: codes and scale bytes bit for bit, products within the bound of
FP32 accumulation."""
import numpy as np
import pytest
import torch

import lowbit_ref as ref
import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import workloads

pytestmark = pytest.mark.gpu
MX, NV = ref.MX, ref.NV
KINDS = [pytest.param(MX, id="mx"), pytest.param(NV, id="nv")]


def gpu(bits):
    return workloads.from_bits(bits).cuda()


def bf16(x):
    """float64 -> BF16 bit patterns."""
    return ref.f64_to_bf16_bits(x)


def data(rows, cols, seed, wide=True):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, cols))
    if wide:
        x *= np.exp(rng.normal(0, 2, (1, cols))) * np.where(rng.random((rows, cols)) < 0.01, 50.0, 1.0)
        x[rng.random((rows, cols)) < 0.02] = 0.0
    return bf16(x)


def check_quant(q, x, kind, t):
    """An Fp4Tensor against the reference of x (float64)."""
    codes, scales = ref.fp4_quant(x, kind, t)
    got_s = q.scales().cpu().numpy()
    assert np.array_equal(got_s, scales), np.argwhere(got_s != scales)[:4]
    packed = q.codes.cpu().numpy()
    want = ref.pack(codes)[:, :(q.k + 1) // 2]
    got = packed[:, :(q.k + 1) // 2]
    # codes that stand for the same value (+0 and -0 are told apart)
    assert np.array_equal(got, want), np.argwhere(got != want)[:4]
    # the padding along k: no scale but 0 reaches the product
    tiled = q.scale.cpu().numpy().reshape(-(-q.rows // 128), -1, 32, 4, 4)
    full = tiled.transpose(0, 3, 2, 1, 4).reshape(tiled.shape[0] * 128, -1)
    assert (full[:q.rows, scales.shape[1]:] == 0).all()


SIZES = [(1, 1), (1, 3584), (2, 15), (3, 17), (5, 32), (7, 255), (16, 256), (33, 257), (128, 128),
         (129, 1003), (200, 512), (300, 96), (1000, 40), (257, 4100), (2, 20000)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quant_rows(cuda_lib, rows, cols, kind):
    bits = data(rows, cols, rows * 7 + cols)
    x = ref.bf16_to_f64(bits)
    t = ref.tensor_scale(x) if kind == NV else 1.0
    ts = torch.tensor([t], device="cuda") if kind == NV else None
    check_quant(fp8hg.fp4_quant(gpu(bits), kind, ts), x, kind, t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quant_both(cuda_lib, rows, cols, kind):
    bits = data(rows, cols, rows * 11 + cols)
    x = ref.bf16_to_f64(bits)
    t = ref.tensor_scale(x) if kind == NV else 1.0
    ts = torch.tensor([t], device="cuda") if kind == NV else None
    q, qt = fp8hg.fp4_quant_dual(gpu(bits), kind, ts)
    check_quant(q, x, kind, t)
    check_quant(qt, x.T, kind, t)
    only = fp8hg.fp4_quant(gpu(bits), kind, ts, transpose=True)
    check_quant(only, x.T, kind, t)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shift,pad", [(0, 0), (8, 8), (1, 0), (3, 5), (0, 3)])
def test_quant_views(cuda_lib, kind, shift, pad):
    """Slices of a wider buffer, aligned and not."""
    bits = data(150, 300 + shift + pad, 5)
    v = gpu(bits)[:, shift:shift + 300]
    x = ref.bf16_to_f64(bits)[:, shift:shift + 300]
    check_quant(fp8hg.fp4_quant(v, kind), x, kind, 1.0)
    q, qt = fp8hg.fp4_quant_dual(v, kind)
    check_quant(q, x, kind, 1.0)
    check_quant(qt, x.T, kind, 1.0)


@pytest.mark.parametrize("kind", KINDS)
def test_quant_special_values(cuda_lib, kind):
    """Blocks with NaN, infinities, zeros, negative zeros, subnormals, the largest values, and midpoints."""
    rng = np.random.default_rng(9)
    bits = data(64, 256, 3)
    bits[0, 5] = 0x7FC0
    bits[1, 40] = 0x7F80
    bits[2, 90] = 0xFF80
    bits[3, :] = 0
    bits[4, :] = 0x8000
    bits[5, :] = rng.integers(0, 0x80, 256)              # subnormals
    bits[6, :] = 0x7F7F
    bits[7, :] = bf16(np.tile([0.25, -0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0, 6.0, 0.0, 5.5, 7.0, -5.0, 1.0, 2.0, 6.0], 16))
    bits[8, :] = bf16(np.tile([1.5, 1e-30], 128))
    x = ref.bf16_to_f64(bits)
    for t in ([1.0] if kind == MX else [1.0, 2.0 ** -7, 2.0 ** 100, 2.0 ** -100]):
        ts = torch.tensor([t], device="cuda") if kind == NV else None
        with np.errstate(over="ignore"):
            q, qt = fp8hg.fp4_quant_dual(gpu(bits), kind, ts)
            check_quant(q, x, kind, t)
            check_quant(qt, x.T, kind, t)
            check_quant(fp8hg.fp4_quant(gpu(bits), kind, ts), x, kind, t)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 3584), (77, 1003), (1000, 4096)])
def test_tensor_scale(cuda_lib, rows, cols):
    bits = data(rows, cols, 21)
    for scale in (1.0, 1e-6, 2.0 ** 20):
        b = bf16(ref.bf16_to_f64(bits) * scale)
        if rows > 1:
            b[0, 0], b[-1, -1] = 0x7F80, 0xFFC0           # left out
        t = fp8hg.fp4_tensor_scale(gpu(b))
        assert t.item() == ref.tensor_scale(ref.bf16_to_f64(b))
    assert fp8hg.fp4_tensor_scale(torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")).item() == 1.0


def test_tensor_scale_at_the_edges(cuda_lib):
    for v in (2688.0, 2704.0, 2672.0, 3.3e38, 1e-38):
        b = bf16(np.array([[v, -v / 2]]))
        assert fp8hg.fp4_tensor_scale(gpu(b)).item() == ref.tensor_scale(ref.bf16_to_f64(b))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 17), (129, 1003), (64, 512)])
def test_dequant(cuda_lib, rows, cols, kind):
    bits = data(rows, cols, 31)
    if cols > 100:
        bits[0, 50] = 0x7FC0
    ts = torch.tensor([0.37], device="cuda") if kind == NV else None
    q = fp8hg.fp4_quant(gpu(bits), kind, ts)
    codes = ref.unpack(q.codes.cpu().numpy(), cols)
    t = float(np.float32(0.37)) if kind == NV else 1.0
    v = ref.fp4_values(codes, q.scales().cpu().numpy(), kind)
    want = (v.astype(np.float32) * np.float32(t)).astype(np.float64) if kind == NV else v
    got = fp8hg.fp4_dequant(q, out_dtype=torch.float32).cpu().numpy().astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)
    # BF16: one rounding of the FP32 value
    b = fp8hg.fp4_dequant(q).float().cpu().numpy().astype(np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(b[fine], ref.bf16_to_f64(bf16(want[fine]))) and np.isnan(b[~fine]).all()
    wide = torch.full((rows, cols + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    fp8hg.fp4_dequant(q, out=wide[:, 1:cols + 1])
    assert np.array_equal(wide[:, 1:cols + 1].float().cpu().numpy(), b.astype(np.float32), equal_nan=True)
    assert (wide[:, 0] == 7).all() and (wide[:, cols + 1:] == 7).all()


# ------------------------------------------------------------------ products
def stored(rows, k, kind, seed, t=None):
    """Random codes and scales as an Fp4Tensor, and their values without t.
    Scales within a few powers of two, so that sums cancel and grow."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    lo, hi = (122, 131) if kind == MX else (0x20, 0x48)
    scales = rng.integers(lo, hi, (rows, -(-k // ref.BLOCK[kind]))).astype(np.uint8)
    ts = torch.tensor([t], dtype=torch.float32, device="cuda") if t is not None else None
    q = fp8hg.Fp4Tensor(torch.from_numpy(ref.pack(codes)).cuda(),
                        torch.from_numpy(ref.tile_scales(scales, k, kind)).cuda(), rows, k, kind, ts)
    return q, torch.from_numpy(ref.fp4_values(codes, scales, kind)).cuda()


def product(a, b):
    """The product and the product of magnitudes, in 64 bits."""
    return (a @ b.t()).cpu().numpy(), (a.abs() @ b.abs().t()).cpu().numpy()


def bound(s_abs, k, ref_c, out):
    """FP32 accumulation over ceil(k / 64) tensor-core steps: each adds its 64
    exact products to the running sum and may lose up to 2^-21 of the largest
    magnitude involved (two bits below FP32's last one); one more rounding per
    scale factor; then one rounding of the output."""
    acc = (-(-k // 64) + 4) * 2.0 ** -21 * s_abs
    return acc + (2.0 ** -8 * np.abs(ref_c) if out == torch.bfloat16 else 2.0 ** -23 * np.abs(ref_c)) + 1e-30


def check_product(got, c, s, k, what=""):
    got = got.detach()
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - c)
    tol = bound(s, k, c, got.dtype)
    assert (err <= tol).all(), (what, float((err / tol).max()), np.argwhere(~(err <= tol))[:4])


SHAPES = [(1, 1, 1), (1, 8, 64), (1, 18944, 3584), (2, 130, 96), (5, 1000, 1536), (8, 256, 256),
          (16, 512, 8960), (17, 129, 255), (33, 1536, 8960), (64, 200, 31), (65, 500, 777), (100, 1, 100),
          (128, 128, 128), (129, 129, 129), (200, 192, 512), (256, 192, 1024), (257, 385, 2048),
          (300, 2048, 640), (640, 1100, 333), (1000, 3584, 1000), (777, 2050, 1999), (2048, 1536, 4096)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(cuda_lib, m, n, k, kind):
    ta, tb = (0.5, 0.3) if kind == NV else (None, None)
    a, va = stored(m, k, kind, m + 3 * n + k, ta)
    b, vb = stored(n, k, kind, m + n + 5 * k, tb)
    c, s = product(va, vb)
    if kind == NV:
        f = float(np.float32(0.5)) * float(np.float32(0.3))
        c, s = c * f, s * f
    check_product(fp8hg.fp4_gemm_scaled(a, b), c, s, k)
    check_product(fp8hg.fp4_gemm_scaled(a, b, out_dtype=torch.float32), c, s, k)
    assert fp8hg.fp8hg_get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", [(1, 300, 640), (40, 130, 512), (300, 500, 512), (129, 777, 65)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_product_accumulates_into_views(cuda_lib, m, n, k, kind, out):
    """C += A B^T into a slice of a wider buffer; nothing beside the slice changes."""
    a, va = stored(m, k, kind, 1)
    b, vb = stored(n, k, kind, 2)
    c, s = product(va, vb)
    for shift in (0, 1, 8):
        wide = torch.randn(m + 2, n + 19, device="cuda").to(out)
        before = wide.clone()
        view = wide[1:m + 1, shift:shift + n]
        fp8hg.fp4_gemm_scaled(a, b, out=view, accumulate=True)
        base = before[1:m + 1, shift:shift + n].double().cpu().numpy()
        check_product(view, base + c, s + np.abs(base), k, shift)
        wide[1:m + 1, shift:shift + n] = before[1:m + 1, shift:shift + n]
        assert torch.equal(wide, before)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(3, 300), (140, 260), (300, 500)])
def test_product_nan_blocks(cuda_lib, m, n, kind):
    """A non-finite block makes its row's (column's) outputs NaN and no others."""
    k = 512
    a, va = stored(m, k, kind, 5)
    b, vb = stored(n, k, kind, 6)
    nan = 0xFF if kind == MX else 0x7F
    a.scale[ref.scale_offset(m - 1, 3, k, kind)] = nan
    b.scale[ref.scale_offset(1, 7, k, kind)] = nan
    got = fp8hg.fp4_gemm_scaled(a, b, out_dtype=torch.float32).cpu().numpy()
    want = np.zeros((m, n), bool)
    want[m - 1, :] = True
    want[:, 1] = True
    assert np.array_equal(np.isnan(got), want)


def test_product_ignores_what_lies_past_the_operands(cuda_lib):
    """Codes past k in a row's padding, scale bytes of rows past the last."""
    for kind in (MX, NV):
        m, n, k = 70, 90, 100
        a, va = stored(m, k, kind, 7)
        b, vb = stored(n, k, kind, 8)
        for q in (a, b):
            q.codes[:, (k + 1) // 2:] = 0x77
            s = q.scale.view(1, -1, 32, 4, 4).permute(0, 3, 2, 1, 4)   # [1, 4, 32, tiles, 4]
            flat = s.reshape(128, -1).clone()
            flat[q.rows:] = 0xFF if kind == MX else 0x7F
            q.scale.copy_(flat.reshape(1, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).reshape(-1))
        c, s = product(va, vb)
        check_product(fp8hg.fp4_gemm_scaled(a, b, out_dtype=torch.float32), c, s, k)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", [(1, 1000, 3584), (1, 5, 18944), (2, 300, 250), (3, 9, 8960), (5, 4000, 300),
                                   (7, 520, 1003), (9, 77, 2000), (16, 256, 512), (17, 40, 5000), (31, 640, 800),
                                   (32, 3, 640), (33, 640, 800), (150, 300, 999), (600, 700, 1024)])
def test_linear_is_quantize_then_multiply(cuda_lib, m, n, k, kind):
    bits = data(m, k, 41)
    if m > 2:
        bits[1, 3] = 0x7FC0
    x = gpu(bits)
    ts = torch.tensor([0.25], device="cuda") if kind == NV else None
    w, vw = stored(n, k, kind, 42, 0.5 if kind == NV else None)
    y = fp8hg.fp4_linear(x, w, ts)
    codes, scales = ref.fp4_quant(ref.bf16_to_f64(bits), kind, 0.25 if kind == NV else 1.0)
    vx = torch.from_numpy(ref.fp4_values(codes, scales, kind)).cuda()
    fine = np.isfinite(ref.bf16_to_f64(bits)).all(1)
    c, s = product(torch.nan_to_num(vx), vw)
    if kind == NV:
        c, s = c * 0.125, s * 0.125
    check_product(y[torch.from_numpy(fine).cuda()], c[fine], s[fine], k)
    assert torch.isnan(y[torch.from_numpy(~fine).cuda()].float()).all()
    # an unaligned view of x gives the same values
    wide = torch.zeros(m, k + 5, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:k + 3] = x
    assert torch.equal(fp8hg.fp4_linear(wide[:, 3:k + 3], w, ts).nan_to_num(), y.nan_to_num())


def test_training_step(cuda_lib):
    """Forward, data gradient and weight gradient of one linear layer from 4-bit operands."""
    m, n, k = 300, 520, 260
    x, w, dy = (ref.bf16_to_f64(data(*s, seed)) for s, seed in (((m, k), 1), ((n, k), 2), ((m, n), 3)))
    for kind in (MX, NV):
        qx, qxt = fp8hg.fp4_quant_dual(gpu(bf16(x)), kind)
        qw, qwt = fp8hg.fp4_quant_dual(gpu(bf16(w)), kind)
        qd, qdt = fp8hg.fp4_quant_dual(gpu(bf16(dy)), kind)
        fq = lambda v: torch.from_numpy(ref.fp4_values(*ref.fp4_quant(v, kind), kind)).cuda()
        for got, a, b, kk in ((fp8hg.fp4_gemm_scaled(qx, qw), fq(x), fq(w), k),
                              (fp8hg.fp4_gemm_scaled(qd, qwt), fq(dy), fq(w.T), n),
                              (fp8hg.fp4_gemm_scaled(qdt, qxt, out_dtype=torch.float32), fq(dy.T), fq(x.T), m)):
            check_product(got, *product(a, b), kk)


def test_repeats_give_the_same_bits_on_other_streams(cuda_lib):
    for kind in (MX, NV):
        for m, n, k in ((1, 700, 3584), (40, 300, 2048), (700, 900, 1100)):
            a, _ = stored(m, k, kind, 11)
            b, _ = stored(n, k, kind, 12)
            want = fp8hg.fp4_gemm_scaled(a, b, out_dtype=torch.float32)
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                outs = [fp8hg.fp4_gemm_scaled(a, b, out_dtype=torch.float32) for _ in range(3)]
            side.synchronize()
            assert all(torch.equal(o, want) for o in outs)


def test_captured_into_a_graph(cuda_lib):
    x = gpu(data(64, 1024, 51))
    w, _ = stored(512, 1024, NV, 52)
    ts = fp8hg.fp4_tensor_scale(x)
    want = fp8hg.fp4_linear(x, w, ts)
    y = torch.empty_like(want)
    ws = torch.empty(fp8hg.fp4_linear_workspace(64, 1024, NV), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8hg.fp4_tensor_scale(x, out=ts)
        fp8hg.fp4_linear(x, w, ts, out=y, workspace=ws)
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_linear_from_several_threads_and_streams(cuda_lib):
    """Calls whose scratch is kept between them: streams of their own, one
    stream shared by two threads, another size each time."""
    import threading
    ws = [stored(300 + 100 * i, 1024, MX, 80 + i)[0] for i in range(3)]
    xs = [gpu(data(8 + 50 * i, 1024, 90 + i)) for i in range(3)]
    want = [[fp8hg.fp4_linear(x, w) for w in ws] for x in xs]
    torch.cuda.synchronize()
    shared, bad = torch.cuda.Stream(), []

    def work(stream):
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = [[fp8hg.fp4_linear(x, w) for w in ws] for x in xs]
        stream.synchronize()
        for i in range(3):
            for j in range(3):
                if not torch.equal(got[i][j], want[i][j]):
                    bad.append((i, j))

    threads = [threading.Thread(target=work, args=(s,)) for s in (shared, shared, torch.cuda.Stream())]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_empty(cuda_lib):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    q = fp8hg.fp4_quant(x, MX)
    w, _ = stored(8, 64, MX, 1)
    assert fp8hg.fp4_gemm_scaled(q, w).shape == (0, 8)
    assert fp8hg.fp4_linear(x, w).shape == (0, 8)
    assert fp8hg.fp4_tensor_scale(x).item() == 1.0


def test_linear_scratch_size(cuda_lib):
    from fp8_hybrid_granularity_gb300 import lowbit
    for kind in (MX, NV):
        for rows, k in ((5, 1), (127, 3584), (129, 257), (1000, 8960)):
            assert lowbit._linear_bytes(rows, k, kind) == fp8hg.fp4_linear_workspace(rows, k, kind)


def test_python_refusals(cuda_lib):
    x = torch.zeros(4, 64, device="cuda")
    w, _ = stored(8, 64, MX, 1)
    for bad in (x, x.bfloat16().cpu(), x.bfloat16().t(), x.bfloat16()[0]):
        with pytest.raises(ValueError):
            fp8hg.fp4_quant(bad, MX)
    with pytest.raises(ValueError):
        fp8hg.fp4_linear(x.bfloat16()[:, :32], w)
    with pytest.raises(ValueError):
        fp8hg.fp4_gemm_scaled(w, w, accumulate=True)
    with pytest.raises(ValueError):
        fp8hg.fp4_gemm_scaled(w, w, out=torch.zeros(8, 9, device="cuda"))
    with pytest.raises(fp8hg.Fp8hgError):
        fp8hg.fp4_gemm_scaled(w, stored(8, 64, NV, 1)[0])
    with pytest.raises(fp8hg.Fp8hgError):
        fp8hg.fp4_quant(x.bfloat16(), MX, torch.ones(1, device="cuda"))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", [(4, 2000, 4096), (100, 400, 2048), (3000, 3000, 1024), (5000, 2304, 4000)])
def test_product_timeout(cuda_lib, m, n, k, kind):
    """A withheld copy and a short limit: the call returns, the status reads
    TIMEOUT once, and the next call is right."""
    a, va = stored(m, k, kind, 61)
    b, vb = stored(n, k, kind, 62)
    fp8hg.fp4_gemm_scaled(a, b, wait_limit_ns=20_000_000, inject_fault=1)
    assert fp8hg.fp8hg_get_device_error() == 6
    assert fp8hg.fp8hg_get_device_error() == 0
    check_product(fp8hg.fp4_gemm_scaled(a, b), *product(va, vb), k)
    assert fp8hg.fp8hg_get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m", [1, 6, 20])
def test_linear_timeout(cuda_lib, m, kind):
    """The product that quantizes its rows itself, with a withheld copy."""
    x = gpu(data(m, 4096, 63))
    w, vw = stored(600, 4096, kind, 64)
    want = fp8hg.fp4_linear(x, w)
    fp8hg.fp4_linear(x, w, wait_limit_ns=20_000_000, inject_fault=1)
    assert fp8hg.fp8hg_get_device_error() == 6
    assert fp8hg.fp8hg_get_device_error() == 0
    assert torch.equal(fp8hg.fp4_linear(x, w), want)


def test_given_stream_owns_what_a_call_allocates(cuda_lib):
    """stream=: results may not land in memory that the current stream still
    has work pending on.  The current stream is held up, writes to a tensor and
    gives its memory back; the call on the other stream then allocates as much."""
    x = gpu(data(512, 2048, 71))
    want = fp8hg.fp4_quant(x, MX)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)
        pending = [torch.empty_like(want.codes).fill_(0xEE), torch.empty_like(want.scale).fill_(0xEE)]
        del pending
        got = fp8hg.fp4_quant(x, MX, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got.codes[:, :1024], want.codes[:, :1024]) and torch.equal(got.scale, want.scale)


# (m, n, k): wide tiles dealt over the machine and a last column of half tiles:
# fewer, one and two rounds of half tiles; one stage of K; a column of exactly
# half a tile; nothing but half tiles next to one wide column
HALF_COLUMNS = [(9000, 2000, 2048), (17900, 480, 2000), (5000, 2112, 250), (20000, 576, 700), (30000, 400, 130),
                (5000, 2400, 4000)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", HALF_COLUMNS)
def test_product_with_a_half_column(cuda_lib, m, n, k, kind):
    """Into views of wider tensors at offsets that TMA can and cannot write:
    the values, and nothing outside."""
    a, va = stored(m, k, kind, 81)
    b, vb = stored(n, k, kind, 82)
    c, s = product(va, vb)
    for dt, off, extra in ((torch.bfloat16, 8, 24), (torch.bfloat16, 3, 9), (torch.float32, 4, 12)):
        wide = torch.full((m + 2, n + extra), 7.0, dtype=dt, device="cuda")
        view = wide[1:m + 1, off:off + n]
        fp8hg.fp4_gemm_scaled(a, b, out=view)
        check_product(view, c, s, k)
        view.fill_(7.0)
        assert bool((wide == 7.0).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(3, 520), (64, 1024), (700, 1536)])
def test_calls_in_a_row_see_each_others_results(cuda_lib, rows, cols, kind):
    """Kernels are launched under the end of the one before: every call of a
    chain without a pause, over the same few buffers, gives what it gives alone."""
    n = 24
    xs = [gpu(data(rows, cols, 900 + i)) for i in range(n)]
    w, _ = stored(256, cols, kind, 91)
    x = torch.empty_like(xs[0])
    ts = torch.ones(1, device="cuda") if kind == NV else None
    q, qt = fp8hg.alloc_fp4(rows, cols, kind), fp8hg.alloc_fp4(cols, rows, kind)

    def chain(src, out):
        x.copy_(src)                       # a kernel that is not the library's
        if kind == NV:
            fp8hg.fp4_tensor_scale(x, out=ts)
        fp8hg.fp4_quant_dual(x, kind, ts, out=q, out_t=qt)
        fp8hg.fp4_dequant(q, out=x)        # in place of its own source
        fp8hg.fp4_dequant(qt, out=out[0])
        fp8hg.fp4_linear(x, w, ts, out=out[1])
        fp8hg.fp4_quant(x, kind, ts, out=q)
        fp8hg.fp4_gemm_scaled(q, w, out=out[2])
        h, _ = fp8hg.fp8_swiglu_ckpt(out[1][:, :128], out[1][:, 128:])
        out[3].copy_(h.codes)

    def outputs():
        e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
        return [e(cols, rows), e(rows, 256), e(rows, 256), torch.empty((rows, 128), dtype=torch.uint8, device="cuda")]
    want = []
    for src in xs:
        want.append(outputs())
        torch.cuda.synchronize()
        chain(src, want[-1])
        torch.cuda.synchronize()
    got = [outputs() for _ in xs]
    torch.cuda.synchronize()
    for src, out in zip(xs, got):
        chain(src, out)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(s.view(torch.uint8), t.view(torch.uint8)) for s, t in zip(a, b))
