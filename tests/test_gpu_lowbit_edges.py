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


# ----------------------------------------------------------- scales far apart
def extreme(rows, k, bytes_, seed, t):
    """An NV tensor of positive values with scale bytes in a range, the first row
    zeros, and its values without t."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(1, 8, (rows, k)).astype(np.uint8)
    codes[0] = 0
    scales = rng.integers(*bytes_, (rows, -(-k // 16))).astype(np.uint8)
    q = fp8hg.Fp4Tensor(torch.from_numpy(ref.pack(codes)).cuda(),
                        torch.from_numpy(ref.tile_scales(scales, k, NV)).cuda(), rows, k, NV,
                        torch.tensor([t], dtype=torch.float32, device="cuda"))
    return q, ref.fp4_values(codes, scales, NV)


HIGH, LOW = (0x70, 0x7F), (0x01, 0x04)     # E4M3 scales of 128 .. 448, of 2^-9 .. 3 2^-9
# tensor scales whose product is 0, subnormal (not a power of two: bits lost), infinite, or in range
PAIRS = [(2.0 ** -75, 2.0 ** -76, HIGH), (1.37 * 2.0 ** -100, 1.21 * 2.0 ** -40, HIGH),
         (2.0 ** 65, 2.0 ** 65, LOW), (2.0 ** 117, 2.0 ** 15, LOW), (2.0 ** 117, 2.0 ** -100, HIGH),
         (1.5 * 2.0 ** -100, 2.0 ** 100, LOW)]


@pytest.mark.parametrize("m,n", [(3, 140), (40, 200), (150, 300), (700, 900), (3000, 2300)])
@pytest.mark.parametrize("ta,tb,bytes_", PAIRS)
def test_tensor_scales_whose_product_leaves_fp32(cuda_lib, m, n, ta, tb, bytes_):
    """Results in FP32's normal range are right wherever the product of the two
    scales lies, and zero rows are zeros.  The sums are within 2^-21 a step of 64
    products (as everywhere in these tests; all products are positive); each scale
    factor and the output round once more."""
    k = 1024 if bytes_ == HIGH else 64
    a, va = extreme(m, k, bytes_, m + n, ta)
    b, vb = extreme(n, k, bytes_, m + n + 1, tb)
    ta, tb = float(np.float32(ta)), float(np.float32(tb))
    c = va @ vb.T
    assert 2.0 ** -125 < c[1:, 1:].min() * ta * tb and c.max() * ta * tb < 2.0 ** 127
    tol = ((k // 64 + 4) * 2.0 ** -21 + 2 * 2.0 ** -24) * c
    for out, ulp in ((torch.float32, 2.0 ** -23), (torch.bfloat16, 2.0 ** -8)):
        got = fp8hg.fp4_gemm_scaled(a, b, out_dtype=out)
        v = got.double().cpu().numpy() / ta / tb
        assert (np.abs(v - c) <= tol + ulp * c).all(), float(np.nanmax(np.abs(v - c) / np.maximum(c, 1e-30)))
        assert not v[0].any() and not v[:, 0].any()
        added = torch.zeros_like(got)
        fp8hg.fp4_gemm_scaled(a, b, out=added, accumulate=True)
        assert torch.equal(added, got)


@pytest.mark.parametrize("value", [2.0 ** 55, 2.0 ** 58])
def test_decoding_with_scales_whose_product_leaves_fp32(cuda_lib, value):
    """x quantized inside the product and before it, tensor scales of 2^65 each:
    rows of zeros give zeros (at 2^55 all are, x's block scales round to 0)."""
    k, t = 512, 2.0 ** 65
    w, vw = extreme(300, k, LOW, 1, t)
    for m in (1, 4, 9):
        x = np.zeros((m, k))
        x[1:] = value
        codes, scales = ref.fp4_quant(x, NV, t)
        c = ref.fp4_values(codes, scales, NV) @ vw.T
        assert c.max() * t * t < 2.0 ** 127 and (m == 1 or c.any() == (value > 2.0 ** 56))
        y = fp8hg.fp4_linear(torch.from_numpy(x).cuda().bfloat16(), w, torch.tensor([t], device="cuda"))
        v = y.double().cpu().numpy() / t / t
        assert (np.abs(v - c) <= ((k // 64 + 4) * 2.0 ** -21 + 2.0 ** -8) * c).all()


def test_largest_tensor_scale(cuda_lib):
    """The scale of a tensor that holds BF16's largest value is 2^117, and the
    quantizer takes it."""
    x = rand(5, 512, 7).float() * 2.0 ** 120
    x[2, 3] = torch.finfo(torch.bfloat16).max
    x = x.bfloat16()
    ts = fp8hg.fp4_tensor_scale(x)
    assert ts.item() == 2.0 ** 117
    codes, scales = ref.fp4_quant(x.double().cpu().numpy(), NV, 2.0 ** 117)
    q, qt = fp8hg.fp4_quant_dual(x, NV, ts)
    assert np.array_equal(q.scales().cpu().numpy(), scales)
    assert np.array_equal(ref.unpack(q.codes.cpu().numpy(), 512), codes)
    codes, scales = ref.fp4_quant(x.t().double().cpu().numpy(), NV, 2.0 ** 117)
    assert np.array_equal(qt.scales().cpu().numpy(), scales)
    assert np.array_equal(ref.unpack(qt.codes.cpu().numpy(), 5), codes)


# ------------------------------------------------- a wait that runs out late
@pytest.mark.parametrize("out,added", [(torch.bfloat16, False), (torch.float32, False), (torch.float32, True),
                                       (torch.bfloat16, True)], ids=["bf16", "f32", "f32-added", "bf16-added"])
def test_wait_that_runs_out_within_a_stage(cuda_lib, out, added):
    """Half of a stage's scales withheld in a pair's second tile, the stages after
    it on their way: the status reads TIMEOUT once, what is stored is right, the tile is
    not stored, and the next call is right.  Added to a C of odd rows the first
    tile is stored long after that wait has begun: the second one's accumulator is
    waited for last."""
    from test_gpu_fp4 import bound, check_product, product, stored
    m, n, k = 9000, 3840, 1024                 # wide tiles, four stages each, five a pair
    a, va = stored(m, k, NV, 101)
    b, vb = stored(n, k, NV, 102)
    c, s = product(va, vb)
    mark = 0.0 if added else float(torch.tensor(1e9).to(out))
    assert np.abs(c).max() < 1e8
    got = torch.empty((m, n + 1), dtype=out, device="cuda")[:, 1:] if added else torch.empty((m, n), dtype=out,
                                                                                            device="cuda")
    tol = bound(s, k, c, out)
    for _ in range(6):
        got.fill_(mark)
        fp8hg.fp4_gemm_scaled(a, b, out=got, accumulate=added, wait_limit_ns=20_000_000, inject_fault=2)
        assert fp8hg.fp8hg_get_device_error() == 6 and fp8hg.fp8hg_get_device_error() == 0
        v = got.double().cpu().numpy()
        wrong = (np.abs(v - c) > tol) & (v != mark)
        assert not wrong.any(), np.argwhere(wrong)[:4]
        assert (v == mark).any()
    got.fill_(0)
    check_product(fp8hg.fp4_gemm_scaled(a, b, out=got, accumulate=added), c, s, k)
    assert fp8hg.fp8hg_get_device_error() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(3, 2000, 4096), (20, 2000, 4096), (50, 700, 8192), (100, 400, 8192), (2500, 2400, 1024)])
def test_nothing_incomplete_is_stored(cuda_lib, m, n, k, out, kind):
    """The first copy withheld: what is stored is right, also by the CTAs that
    share a tile's K with the one that waited in vain."""
    from test_gpu_fp4 import bound, product, stored
    a, va = stored(m, k, kind, 161)
    b, vb = stored(n, k, kind, 162)
    c, s = product(va, vb)
    mark = float(torch.tensor(1e9).to(out))
    got = torch.full((m, n), mark, dtype=out, device="cuda")
    fp8hg.fp4_gemm_scaled(a, b, out=got, wait_limit_ns=20_000_000, inject_fault=1)
    assert fp8hg.fp8hg_get_device_error() == 6
    v = got.double().cpu().numpy()
    wrong = (np.abs(v - c) > bound(s, k, c, out)) & (v != mark)
    assert not wrong.any(), np.argwhere(wrong)[:4]
    assert (v == mark).any()


def test_fault_that_a_shape_cannot_have(cuda_lib):
    from test_gpu_fp4 import stored
    for kind, status in ((MX, 1), (NV, 4)):
        a, b = stored(3, 64, kind, 1)[0], stored(40, 64, kind, 2)[0]
        with pytest.raises(fp8hg.Fp8hgError) as e:
            fp8hg.fp4_gemm_scaled(a, b, inject_fault=2)
        assert e.value.status == status
    with pytest.raises(fp8hg.Fp8hgError):
        fp8hg.fp4_linear(rand(9, 64, 1), b, inject_fault=2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(1000, 3584), (2048, 2300)])
def test_product_of_a_long_k(cuda_lib, m, n, kind):
    """74 stages of K in the kernels of larger products."""
    from test_gpu_fp4 import check_product, product, stored
    k = 18944
    a, va = stored(m, k, kind, 111)
    b, vb = stored(n, k, kind, 112)
    check_product(fp8hg.fp4_gemm_scaled(a, b, out_dtype=torch.float32), *product(va, vb), k)


# ------------------------------------------------------------------ long axes
LONG = 65536 * 4096 + 3 * 4096 + 304      # columns: more chunks of 4096 than a grid has in its second dimension


def folded(x):
    """The whole chunks of 4096 columns of a few long rows, as rows of 4096."""
    return x[:, :LONG // 4096 * 4096].reshape(-1, 4096)


@pytest.mark.parametrize("kind", KINDS)
def test_quantizer_of_very_long_rows(cuda_lib, kind):
    """Two rows of 2^28 columns and more, against the same data in short rows."""
    x = rand(2, LONG, 121)
    q, short = fp8hg.fp4_quant(x, kind), fp8hg.fp4_quant(folded(x).contiguous(), kind)
    assert torch.equal(folded(q.codes.repeat_interleave(2, 1)[:, :LONG])[:, ::2], short.codes)
    n = 4096 // ref.BLOCK[kind]
    whole = LONG // 4096 * n
    assert torch.equal(q.scales()[:, :whole].reshape(-1, n), short.scales())
    tail = fp8hg.fp4_quant(x[:, whole * ref.BLOCK[kind]:], kind)
    assert torch.equal(q.scales()[:, whole:], tail.scales())
    v = fp8hg.fp4_dequant(q)
    assert torch.equal(folded(v), fp8hg.fp4_dequant(short))
    assert torch.equal(v[:, whole * ref.BLOCK[kind]:], fp8hg.fp4_dequant(tail))
    del v
    assert torch.equal(folded(fp8hg.fp4_dequant(q, out_dtype=torch.float32)),
                       fp8hg.fp4_dequant(short, out_dtype=torch.float32))


def test_swiglu_of_very_long_rows(cuda_lib):
    g, u, dh = (rand(2, LONG, 131 + i) for i in range(3))
    cut = LONG // 4096 * 4096
    h, ck = fp8hg.fp8_swiglu_ckpt(g, u)
    parts = [[folded(t).contiguous() for t in (g, u, dh)], [t[:, cut:] for t in (g, u, dh)]]
    d = fp8hg.fp8_swiglu_ckpt_bwd(dh, ck)
    halves = [d[:, :LONG], d[:, LONG:]]
    for i, (pg, pu, pdh) in enumerate(parts):
        at = (lambda t: t[:, cut:]) if i else folded
        ats = (lambda s: s[:, cut // 128:]) if i else lambda s: s[:, :cut // 128].reshape(-1, 32)
        ph, pck = fp8hg.fp8_swiglu_ckpt(pg, pu)
        for a, b in ((h, ph), (ck.gate, pck.gate), (ck.up, pck.up)):
            assert torch.equal(at(a.codes), b.codes) and torch.equal(ats(a.scales()), b.scales())
        pd = fp8hg.fp8_swiglu_ckpt_bwd(pdh, pck)
        n = pdh.shape[1]
        assert torch.equal(at(halves[0]), pd[:, :n]) and torch.equal(at(halves[1]), pd[:, n:])


def test_most_rows_of_the_quantizer_along_the_columns(cuda_lib):
    """As many rows as are taken; one more is refused, and the refusal leaves nothing behind."""
    rows = 32767 * 256
    x = rand(rows + 1, 32, 141)
    with pytest.raises(fp8hg.Fp8hgError) as e:
        fp8hg.fp4_quant(x, MX, transpose=True)
    assert e.value.status == 3
    fp8hg.fp8_quant_token(rand(128, 128, 142))
    for kind in (MX, NV):
        q, qt = fp8hg.fp4_quant_dual(x[:rows], kind)
        assert torch.equal(q.codes, fp8hg.fp4_quant(x[:rows], kind).codes)
        s = qt.scales()
        for at in (0, 12345 * 256, rows - 256):
            part = fp8hg.fp4_quant(x[at:at + 256], kind, transpose=True)
            assert torch.equal(qt.codes[:, at // 2:at // 2 + 128], part.codes)
            n = ref.BLOCK[kind]
            assert torch.equal(s[:, at // n:at // n + 256 // n], part.scales())


def test_many_rows_of_the_swiglu_backward(cuda_lib):
    """More rows than a grid's second dimension would hold in tiles, and rows that
    the CTAs of a column step through."""
    rows = 65536 * 128 + 128
    g, u, dh = (rand(rows, 128, 151 + i) for i in range(3))
    h, ck = fp8hg.fp8_swiglu_ckpt(g, u)
    d = fp8hg.fp8_swiglu_ckpt_bwd(dh, ck)
    dq, dt, ht = fp8hg.fp8_swiglu_ckpt_bwd_q(dh, ck)
    for at in (0, 70000 * 64, rows - 128):
        r = slice(at, at + 128)
        ph, pck = fp8hg.fp8_swiglu_ckpt(g[r], u[r])
        assert torch.equal(h.codes[r], ph.codes) and torch.equal(ck.gate.codes[r], pck.gate.codes)
        assert torch.equal(d[r], fp8hg.fp8_swiglu_ckpt_bwd(dh[r], pck))
        a, b, c = fp8hg.fp8_swiglu_ckpt_bwd_q(dh[r], pck)
        assert torch.equal(dq.codes[r], a.codes) and torch.equal(dq.scales()[r], a.scales())
        assert torch.equal(dt.codes[:, r], b.codes) and torch.equal(ht.codes[:, r], c.codes)
        assert torch.equal(ht.scales()[:, at // 128:at // 128 + 1], c.scales())
    assert fp8hg.fp8hg_get_device_error() == 0
