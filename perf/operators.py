"""Cases for measuring the 4-bit operators and the SwiGLU with 8-bit checkpoints.

Every case runs in two forms on the same inputs: the plain one (`own` false),
elementary torch operations in 32 bits, and the framework's own kernels
(`own` true), through its public Python functions.  The operators:

  quant       BF16 -> E2M1 codes with MX (32 elements, power-of-two) or NV
              (16 elements, E4M3 and one FP32 scale per tensor) block scales,
              along the rows or along rows and columns, and back to values
  linear      y = x w^T with x quantized in the call and w stored in 4 bits
  linear_bwd  dx = dy w, dw = dy^T x with dy quantized in both directions
  swiglu      h = silu(gate) * up in FP8, gate and up kept as 8-bit checkpoints
  swiglu_bwd  gradients of gate and up from dh and the checkpoints, in BF16, or
              in FP8 in both directions together with the rebuilt h

Layer sizes are those of the 1.5B (hidden 1536, MLP 8960) and 7B (hidden 3584,
MLP 18944) layers that the benchmark of this repository runs.
"""
import math

import torch

own = False

MX, NV = "mx", "nv"
BLOCK = {MX: 32, NV: 16}


def listed():
    return [
        # the hidden activation of the 1.5B layer for a training step: the tensor's scale, then both directions
        dict(name="quant_nv_both_8192x8960", op="quant", kind=NV, both=True, rows=8192, cols=8960, pad=0),
        # an odd slice out of a wider buffer, rows only
        dict(name="quant_mx_rows_1111x1003", op="quant", kind=MX, both=False, rows=1111, cols=1003, pad=37),
        # decoding: one token through the 7B layer's gate projection
        dict(name="linear_nv_1x18944x3584", op="linear", kind=NV, m=1, n=18944, k=3584),
        # decoding a batch through the 1.5B layer's down projection
        dict(name="linear_mx_33x1536x8960", op="linear", kind=MX, m=33, n=1536, k=8960),
        # a short prompt, sizes that fill no tile
        dict(name="linear_mx_777x2050x1999", op="linear", kind=MX, m=777, n=2050, k=1999),
        # a long prompt (or the forward of a training step), 7B gate projection
        dict(name="linear_nv_8192x18944x3584", op="linear", kind=NV, m=8192, n=18944, k=3584),
        # training: the backward of the 1.5B gate projection
        dict(name="linear_bwd_mx_8192x8960x1536", op="linear_bwd", kind=MX, m=8192, n=8960, k=1536),
        # the backward of the 7B down projection over a short batch
        dict(name="linear_bwd_nv_1000x3584x18944", op="linear_bwd", kind=NV, m=1000, n=3584, k=18944),
        # the MLP of a few decoded tokens, 1.5B layer
        dict(name="swiglu_37x8960", op="swiglu", rows=37, cols=8960),
        # a training step of the 7B layer
        dict(name="swiglu_16384x18944", op="swiglu", rows=16384, cols=18944),
        # the backward of the 1.5B layer's training step, ready for the FP8 products
        dict(name="swiglu_bwd_q_8192x8960", op="swiglu_bwd", quantized=True, rows=8192, cols=8960),
        # sizes that fill no group, BF16 gradients
        dict(name="swiglu_bwd_1500x5001", op="swiglu_bwd", quantized=False, rows=1500, cols=5001),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "linear_bwd", "swiglu", "swiglu_bwd"])
    if op == "quant":
        return dict(op=op, kind=rng.choice([MX, NV]), both=rng.random() < 0.5, rows=_spread(rng, 16, 8192),
                    cols=_spread(rng, 512, 8960), pad=rng.choice([0, 8, 37]))
    if op == "linear":
        return dict(op=op, kind=rng.choice([MX, NV]), m=_spread(rng, 1, 8192), n=_spread(rng, 512, 18944),
                    k=_spread(rng, 512, 3584) if rng.random() < 0.5 else rng.choice([1536, 2048, 3584]))
    if op == "linear_bwd":
        return dict(op=op, kind=rng.choice([MX, NV]), m=_spread(rng, 64, 8192), n=_spread(rng, 512, 8960),
                    k=rng.choice([1536, 3584]) if rng.random() < 0.5 else _spread(rng, 512, 3584))
    if op == "swiglu":
        return dict(op=op, rows=_spread(rng, 1, 16384), cols=_spread(rng, 512, 18944))
    quantized = rng.random() < 0.5
    rows, cols = _spread(rng, 128, 8192), _spread(rng, 512, 8960)
    if quantized:  # the FP8 products take multiples of 128
        rows, cols = -(-rows // 128) * 128, -(-cols // 128) * 128
    return dict(op=op, quantized=quantized, rows=rows, cols=cols)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _act(g, rows, cols):
    """Activations: channels of different ranges and a few strong outliers."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(1, cols, generator=g, device="cuda"))
    x *= torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 1e-3, 30.0, 1.0)
    return x.bfloat16()


def _grad(g, rows, cols):
    """Gradients: small, with heavy tails (Student's t, three degrees of freedom)."""
    z = torch.randn(rows, cols, generator=g, device="cuda")
    c = torch.zeros(rows, cols, device="cuda")
    for _ in range(3):
        c += torch.randn(rows, cols, generator=g, device="cuda").square_()
    return (1e-3 * z / (c / 3).sqrt()).bfloat16()


def _stored(x, kind):
    """A weight or a kept activation as a program stores it: packed codes (rows
    padded to 16 bytes), block scales in 128-row tiles, the tensor's scale."""
    t = _tensor_scale(x) if kind == NV else None
    codes, scales = _quantize(x, kind, t)
    return dict(codes=_pack(codes), scale=_tile_scales(scales, kind), tensor_scale=t, rows=x.shape[0], k=x.shape[1])


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "quant":
        x = _act(g, case["rows"], case["cols"] + case["pad"])
        s["x"] = x[:, case["pad"]:]
    elif op == "linear":
        s["x"] = _act(g, case["m"], case["k"])
        s["w"] = _stored((0.02 * torch.randn(case["n"], case["k"], generator=g, device="cuda")).bfloat16(), case["kind"])
        # calibrated beforehand, as for serving
        s["x_scale"] = torch.full((1,), 0.5, device="cuda") if case["kind"] == NV else None
    elif op == "linear_bwd":
        s["dy"] = _grad(g, case["m"], case["n"])
        s["x_t"] = _stored(_act(g, case["m"], case["k"]).t().contiguous(), case["kind"])
        w = (0.02 * torch.randn(case["n"], case["k"], generator=g, device="cuda")).bfloat16()
        s["w_t"] = _stored(w.t().contiguous(), case["kind"])
    else:
        rows, cols = case["rows"], case["cols"]
        gate_up = torch.randn(rows, 2 * cols, generator=g, device="cuda")
        gate_up *= torch.exp(0.5 * torch.randn(1, 2 * cols, generator=g, device="cuda"))
        gate_up = gate_up.bfloat16()
        if op == "swiglu":
            s["gate"], s["up"] = gate_up[:, :cols], gate_up[:, cols:]   # one product wrote both
        else:
            for name, part in (("gate", gate_up[:, :cols]), ("up", gate_up[:, cols:])):
                q, e = _fp8_groups(part.float(), torch.float8_e4m3fn)
                codes = torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda")
                codes[:, :cols] = q.view(torch.uint8)
                scale = torch.zeros(rows, -(-e.shape[1] // 4) * 4, dtype=torch.uint8, device="cuda")
                scale[:, :e.shape[1]] = (e + 127).to(torch.uint8)
                s[name + "_codes"], s[name + "_scale"] = codes[:, :cols], scale
            s["dh"] = _grad(g, rows, cols)
    return s


# ---------------------------------------------------------------- plain forms
def _blocks(x, n):
    """[rows, cols] as [rows, blocks, n], zeros after the last column."""
    rows, cols = x.shape
    nb = -(-cols // n)
    if nb * n != cols:
        x = torch.nn.functional.pad(x, (0, nb * n - cols))
    return x.reshape(rows, nb, n)


def _e2m1(v):
    """Codes of the nearest E2M1 values, ties to the even code, at most 6."""
    a = v.abs()
    c = (a > 0.25).to(torch.uint8)
    c += a >= 0.75
    c += a > 1.25
    c += a >= 1.75
    c += a > 2.5
    c += a >= 3.5
    c += a > 5.0
    return c + 8 * torch.signbit(v).to(torch.uint8)


def _tensor_scale(x):
    """The smallest power of two t with amax <= 6 * 448 * t."""
    m, e = torch.frexp(x.abs().amax().float())
    t = torch.ldexp(torch.ones_like(m), e - 12 + (m > 0.65625).int())
    return torch.where(m > 0, t, torch.ones_like(t)).reshape(1)


def _quantize(x, kind, tensor_scale):
    """Codes [rows, cols] and scale bytes [rows, blocks]."""
    b = _blocks(x.float(), BLOCK[kind])
    amax = b.abs().amax(2)
    if kind == MX:
        e = (torch.frexp(amax)[1].clamp(-1000, 1000) - 3).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        codes = _e2m1(torch.ldexp(b, -e.unsqueeze(2)))
        scales = (e + 127).to(torch.uint8)
    else:
        s = ((amax / 6.0) / tensor_scale).clamp(max=448.0).to(torch.float8_e4m3fn)
        f = s.float()
        d = torch.where(f > 0, f * tensor_scale, torch.full_like(f, math.inf))
        codes = _e2m1(b / d.unsqueeze(2))
        scales = s.view(torch.uint8)
    return codes.reshape(x.shape[0], -1)[:, :x.shape[1]], scales


def _power(byte):
    return torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.int() - 127)


def _values(codes, scales, kind):
    """Codes times block scales, in 32 bits; the tensor's scale is left out."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    s = _power(scales) if kind == MX else scales.view(torch.float8_e4m3fn).float()
    v = _blocks(table[codes.int()], BLOCK[kind]) * s.unsqueeze(2)
    return v.reshape(codes.shape[0], -1)[:, :codes.shape[1]]


def _pack(codes):
    rows, cols = codes.shape
    ld = -(-cols // 32) * 16
    p = torch.zeros(rows, 2 * ld, dtype=torch.uint8, device=codes.device)
    p[:, :cols] = codes
    return p[:, 0::2] | (p[:, 1::2] << 4)


def _unpack(p, cols):
    return torch.stack([p & 15, p >> 4], 2).reshape(p.shape[0], -1)[:, :cols]


def _tile_scales(s, kind):
    """Scale bytes in tiles of 128 rows by 4 blocks, 512 bytes each, the tiles of
    128 rows after one another; within a tile row r comes at 16 (r mod 32) + 4 (r / 32)."""
    per = 256 // BLOCK[kind]
    rows, n = s.shape
    r, b = -(-rows // 128), -(-n // per) * per // 4
    t = torch.zeros(r * 128, b * 4, dtype=torch.uint8, device=s.device)
    t[:rows, :n] = s
    return t.reshape(r, 4, 32, b, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile_scales(t, rows, k, kind):
    n = -(-k // BLOCK[kind])
    per = 256 // BLOCK[kind]
    r, b = -(-rows // 128), -(-n // per) * per // 4
    return t.reshape(r, b, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, b * 4)[:rows, :n]


def _stored_values(w, kind):
    return _values(_unpack(w["codes"], w["k"]), _untile_scales(w["scale"], w["rows"], w["k"], kind), kind)


def _scaled(v, *scales):
    f = None
    for s in scales:
        if s is not None:
            f = s if f is None else f * s
    return v if f is None else v * f


def _fp8_groups(x, dtype):
    """FP8 codes [rows, cols] and exponents [rows, groups of 128 columns], the
    smallest power of two that keeps the group within the format."""
    b = _blocks(x, 128)
    m, e = torch.frexp(b.abs().amax(2))
    e = e - (9 if dtype == torch.float8_e4m3fn else 16) + (m > 0.875).int()
    e = torch.where(m > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    q = torch.ldexp(b, -e.unsqueeze(2)).reshape(x.shape[0], -1)[:, :x.shape[1]]
    return q.to(dtype), e


def _fp8_out(x, dtype):
    q, e = _fp8_groups(x, dtype)
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _fp8_values(codes, scale):
    cols = codes.shape[1]
    s = _power(scale)
    v = _blocks(codes.view(torch.float8_e4m3fn).float(), 128)
    return (v * s[:, :v.shape[1]].unsqueeze(2)).reshape(codes.shape[0], -1)[:, :cols]


def _plain(s):
    op = s["op"]
    if op == "quant":
        x, kind = s["x"], s["kind"]
        t = _tensor_scale(x) if kind == NV else None
        out = [_scaled(_values(*_quantize(x, kind, t), kind), t).bfloat16()]
        if s["both"]:
            out.append(_scaled(_values(*_quantize(x.t(), kind, t), kind), t).bfloat16())
        return out
    if op == "linear":
        kind = s["kind"]
        x = _values(*_quantize(s["x"], kind, s["x_scale"]), kind)
        return _scaled(x @ _stored_values(s["w"], kind).t(), s["x_scale"], s["w"]["tensor_scale"]).bfloat16()
    if op == "linear_bwd":
        kind, dy = s["kind"], s["dy"]
        t = _tensor_scale(dy) if kind == NV else None
        d = _values(*_quantize(dy, kind, t), kind)
        dx = _scaled(d @ _stored_values(s["w_t"], kind).t(), t, s["w_t"]["tensor_scale"]).bfloat16()
        d = _values(*_quantize(dy.t(), kind, t), kind)
        return dx, _scaled(d @ _stored_values(s["x_t"], kind).t(), t, s["x_t"]["tensor_scale"]).bfloat16()
    if op == "swiglu":
        gate, up = s["gate"].float(), s["up"].float()
        h = gate / (1 + torch.exp(-gate)) * up
        return [_fp8_out(v, torch.float8_e4m3fn) for v in (h, gate, up)]
    gate, up, dh = _fp8_values(s["gate_codes"], s["gate_scale"]), _fp8_values(s["up_codes"], s["up_scale"]), s["dh"].float()
    sig = 1 / (1 + torch.exp(-gate))
    d = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1)
    if not s["quantized"]:
        return d.bfloat16()
    h = gate * sig * up
    return [_fp8_out(d, torch.float8_e5m2), _fp8_out(d.t().contiguous(), torch.float8_e5m2), _fp8_out(h.t().contiguous(), torch.float8_e4m3fn)]


# ---------------------------------------------------------------- the framework's operators
_FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)


def _shown(q):
    """An FP8 tensor's codes and scale bytes as the numbers they are."""
    return q.codes.view(_FP8[q.fmt]), q.scales().view(torch.float8_e8m0fnu)


def _framework(s):
    import fp8_hybrid_granularity_gb300 as hg
    op = s["op"]
    kind = {MX: hg.FP4_MX, NV: hg.FP4_NV}.get(s.get("kind"))

    def stored(w):
        return hg.Fp4Tensor(w["codes"], w["scale"], w["rows"], w["k"], kind, w["tensor_scale"])

    if op == "quant":
        x = s["x"]
        t = hg.fp4_tensor_scale(x) if kind == hg.FP4_NV else None
        if s["both"]:
            return [hg.fp4_dequant(q) for q in hg.fp4_quant_dual(x, kind, t)]
        return [hg.fp4_dequant(hg.fp4_quant(x, kind, t))]
    if op == "linear":
        return hg.fp4_linear(s["x"], stored(s["w"]), s["x_scale"])
    if op == "linear_bwd":
        dy = s["dy"]
        d, d_t = hg.fp4_quant_dual(dy, kind, hg.fp4_tensor_scale(dy) if kind == hg.FP4_NV else None)
        return hg.fp4_gemm_scaled(d, stored(s["w_t"])), hg.fp4_gemm_scaled(d_t, stored(s["x_t"]))
    if op == "swiglu":
        h, kept = hg.fp8_swiglu_ckpt(s["gate"], s["up"])
        return [_shown(q) for q in (h, kept.gate, kept.up)]
    groups = -(-s["cols"] // 128)
    kept = hg.SwigluCkpt(*(hg.QTensor(s[n + "_codes"], s[n + "_scale"], hg.E4M3, hg.GRAN_1x128, groups) for n in ("gate", "up")))
    if not s["quantized"]:
        return hg.fp8_swiglu_ckpt_bwd(s["dh"], kept)
    return [_shown(q) for q in hg.fp8_swiglu_ckpt_bwd_q(s["dh"], kept)]


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def _fp4_bytes(rows, k, kind):
    return rows * (-(-k // 2) + -(-k // BLOCK[kind]))


def work(case):
    op = case["op"]
    if op == "quant":  # x in; codes, scales and values out
        n = case["rows"] * case["cols"]
        out = _fp4_bytes(case["rows"], case["cols"], case["kind"]) + 2 * n
        if case["both"]:
            out += _fp4_bytes(case["cols"], case["rows"], case["kind"]) + 2 * n
        return {"bytes": 2 * n + out, "flops": 0}
    if op in ("linear", "linear_bwd"):
        m, n, k, kind = case["m"], case["n"], case["k"], case["kind"]
        if op == "linear":
            return {"bytes": 2 * m * k + _fp4_bytes(n, k, kind) + 2 * m * n, "flops": 2 * m * n * k}
        return {"bytes": 2 * m * n + _fp4_bytes(k, m, kind) + _fp4_bytes(k, n, kind) + 2 * m * k + 2 * n * k, "flops": 4 * m * n * k}
    n = case["rows"] * case["cols"]
    if op == "swiglu":
        return {"bytes": 4 * n + 3 * n + 3 * n // 128, "flops": 0}
    out = 5 * n + 5 * n // 128 if case["quantized"] else 4 * n
    return {"bytes": 2 * n + 2 * n + 2 * n // 128 + out, "flops": 0}


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _floor_log2(a):
    """Exponent of the largest power of two that is not above a > 0 (a logarithm could round across it)."""
    return (torch.frexp(a.clamp(min=2.0 ** -1000))[1] - 1).double()


def _round64(v, top, least):
    """Nearest value of a small floating format: two or more mantissa steps per
    power of two (`least`: smallest exponent, steps), ties to even, at most `top`."""
    emin, steps = least
    step = torch.exp2(_floor_log2(v.abs()).clamp(min=emin)) / steps
    return (torch.round(v / step) * step).clamp(-top, top)


def _fq64(x, kind, t):
    """x rounded to 4 bits and back, without the tensor's scale."""
    rows, cols = x.shape
    n = BLOCK[kind]
    out = torch.zeros(rows, -(-cols // n) * n, dtype=torch.float64, device=x.device)
    out[:, :cols] = x
    b = out.view(rows, -1, n)
    top = b.abs().amax(2, keepdim=True)
    if kind == MX:
        s = torch.exp2((_floor_log2(top) - 2).clamp(min=-127))
        b = _round64(b / s, 6.0, (0, 2)) * s
    else:
        s = _round64(top / (6 * t), 448.0, (-6, 8))
        b = torch.where(s > 0, _round64(b / (s * t).clamp(min=1e-300), 6.0, (0, 2)) * s, torch.zeros_like(b))
    return b.reshape(rows, -1)[:, :cols]


def _t64(x):
    need = x.abs().max().double() / 2688
    e = _floor_log2(need)
    return torch.exp2(e + (need > torch.exp2(e))) if need > 0 else need + 1


def _stored64(w, kind):
    """Read byte by byte: where a block's scale lies follows from the tile's description."""
    rows, k = w["rows"], w["k"]
    dev = w["codes"].device
    per_tile = -(-k // 256) * (256 // BLOCK[kind]) // 4
    r = torch.arange(rows, device=dev).unsqueeze(1)
    j = torch.arange(-(-k // BLOCK[kind]), device=dev).unsqueeze(0)
    byte = w["scale"][((r // 128) * per_tile + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4].long()
    if kind == MX:
        s = torch.exp2(byte.double() - 127)
    else:
        e, m = byte >> 3, (byte & 7).double()
        s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6)
    i = torch.arange(k, device=dev)
    c = (w["codes"][:, i // 2] >> (4 * (i % 2)).to(torch.uint8)) & 15
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e.double() - 1), m / 2)
    v = torch.where(c >= 8, -v, v)
    return v * s.repeat_interleave(BLOCK[kind], 1)[:, :k]


def _fp8_64(x, fmt):
    """FP8 codes' values and the scales' values of groups of 128 columns."""
    top, emin, steps = (448.0, -6, 8) if fmt == torch.float8_e4m3fn else (57344.0, -14, 4)
    rows, cols = x.shape
    g = -(-cols // 128)
    b = torch.zeros(rows, g * 128, dtype=torch.float64, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, g, 128)
    need = b.abs().amax(2) / top
    e = _floor_log2(need)
    s = torch.exp2((e + (need > torch.exp2(e))).clamp(-127, 127))
    q = _round64(b / s.unsqueeze(2), top, (emin, steps)).reshape(rows, -1)[:, :cols]
    return q, s


def _e4m3_64(codes, scale):
    c = codes.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m / 8 * 2.0 ** -6)
    v = torch.where(c >= 128, -v, v)
    return v * torch.exp2(scale.double() - 127).repeat_interleave(128, 1)[:, :codes.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    op, kind = case["op"], case.get("kind")
    if op == "quant":
        x = s["x"].double()
        t = _t64(x) if kind == NV else 1.0
        return [_fq64(v, kind, t) * t for v in ([x, x.t()] if case["both"] else [x])]
    if op == "linear":
        t = s["x_scale"].double() if kind == NV else 1.0
        u = s["w"]["tensor_scale"].double() if kind == NV else 1.0
        return _fq64(s["x"].double(), kind, t) @ _stored64(s["w"], kind).t() * t * u
    if op == "linear_bwd":
        dy = s["dy"].double()
        t = _t64(dy) if kind == NV else 1.0
        u, v = (s[n]["tensor_scale"].double() if kind == NV else 1.0 for n in ("w_t", "x_t"))
        return (_fq64(dy, kind, t) @ _stored64(s["w_t"], kind).t() * t * u, _fq64(dy.t(), kind, t) @ _stored64(s["x_t"], kind).t() * t * v)
    if op == "swiglu":
        gate, up = s["gate"].double(), s["up"].double()
        return [_fp8_64(v, torch.float8_e4m3fn) for v in (gate * torch.sigmoid(gate) * up, gate, up)]
    gate, up, dh = _e4m3_64(s["gate_codes"], s["gate_scale"]), _e4m3_64(s["up_codes"], s["up_scale"]), s["dh"].double()
    sig = torch.sigmoid(gate)
    d = torch.cat([dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig], 1)
    if not case["quantized"]:
        return d
    return [_fp8_64(d, torch.float8_e5m2), _fp8_64(d.t(), torch.float8_e5m2), _fp8_64((gate * sig * up).t(), torch.float8_e4m3fn)]
