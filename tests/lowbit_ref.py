"""Plain 64-bit references of the 4-bit operators and of the SwiGLU with 8-bit
checkpoints, in numpy, written from the formats' definitions: values are looked
up in tables of all codes, roundings are nearest-value searches."""
from __future__ import annotations

import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
E4M3, E5M2 = 0, 1

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _fp8_table(fmt):
    """Values of the non-negative finite codes in code order."""
    v = []
    for c in range(0x7F if fmt == E4M3 else 0x7C):
        if fmt == E4M3:
            e, m = c >> 3, c & 7
            v.append((1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6)
        else:
            e, m = c >> 2, c & 3
            v.append((1 + m / 4) * 2.0 ** (e - 15) if e else m / 4 * 2.0 ** -14)
    return np.array(v)


FP8 = {E4M3: _fp8_table(E4M3), E5M2: _fp8_table(E5M2)}


def nearest(table, a):
    """Index of the nearest entry of an ascending table to a >= 0, ties to the
    even index, the last entry beyond the end."""
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(a >= table[-1], len(table) - 1, np.where(up, hi, lo))


def bf16_to_f64(bits):
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


def f64_to_bf16_bits(x):
    """Round to nearest even (finite values)."""
    f = np.asarray(x, np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def tensor_scale(x):
    """The smallest power of two t >= 2^-100 with amax of the finite values <= 2688 t."""
    x = x[np.isfinite(x)]
    a = np.abs(x).max() if x.size else 0.0
    if a == 0:
        return 1.0
    t = 2.0 ** -100
    while a > 2688 * t:
        t *= 2
    return t


def fp4_quant(x, kind, t=1.0):
    """x [rows, cols] float64 -> codes [rows, cols] uint8, scale bytes [rows, blocks]."""
    rows, cols = x.shape
    n = BLOCK[kind]
    nb = -(-cols // n)
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    for j in range(nb):
        b = x[:, j * n:(j + 1) * n]
        bad = ~np.isfinite(b).all(1)
        b = np.where(bad[:, None], 0.0, b)
        amax = np.abs(b).max(1)
        if kind == MX:
            e = np.where(amax > 0, np.frexp(np.where(amax > 0, amax, 1.0))[1] - 3, -127)
            e = np.clip(e, -127, 127)
            v = b / np.exp2(e.astype(np.float64))[:, None]
            s = np.where(bad, 0xFF, e + 127)
        else:
            # the two quotients are rounded to FP32, as the definition says
            q = np.float32(np.float32(amax) / np.float32(6)) / np.float32(t)
            s = nearest(FP8[E4M3], q)
            d = FP8[E4M3][s] * t
            v = np.where(d[:, None] > 0, b / np.where(d > 0, d, 1.0)[:, None], 0.0)
            s = np.where(bad, 0x7F, s)
        # the sign of zero: MX keeps it, NV codes -0 as 0
        c = nearest(E2M1, np.abs(v)) | ((np.signbit(b) if kind == MX else b < 0) * 8)
        codes[:, j * n:(j + 1) * n] = np.where(bad[:, None], 0, c)
        scales[:, j] = s
    return codes, scales


def scale_values(scales, kind):
    s = scales.astype(int)
    if kind == MX:
        return np.where(s == 0xFF, np.nan, np.exp2(s - 127.0))
    return np.where(s == 0x7F, np.nan, FP8[E4M3][np.minimum(s, 0x7E)])


def fp4_values(codes, scales, kind, t=1.0):
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.repeat(scale_values(scales, kind), BLOCK[kind], 1)[:, :codes.shape[1]]
    return v * s * t


def pack(codes):
    rows, cols = codes.shape
    p = np.zeros((rows, -(-cols // 32) * 32), np.uint8)
    p[:, :cols] = codes
    return p[:, 0::2] | (p[:, 1::2] << 4)


def unpack(packed, cols):
    return np.stack([packed & 15, packed >> 4], 2).reshape(packed.shape[0], -1)[:, :cols]


def scale_offset(r, j, k, kind):
    tiles = -(-k // 256) * (4 if kind == NV else 2)
    return ((r // 128) * tiles + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4


def tile_scales(scales, k, kind):
    rows, nb = scales.shape
    size = -(-rows // 128) * (-(-k // 256)) * (4 if kind == NV else 2) * 512
    t = np.zeros(size, np.uint8)
    r, j = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    t[scale_offset(r, j, k, kind)] = scales
    return t


# ------------------------------------------------------------------- SwiGLU
def ue8m0(amax, fmt):
    """Smallest e in [-127, 127] with amax <= FMAX 2^e."""
    top = 448.0 if fmt == E4M3 else 57344.0
    m, e = np.frexp(np.where(amax > 0, amax, 1.0) / top)
    e = np.where(m > 0.5, e, e - 1)
    return np.clip(np.where(amax > 0, e, -127), -127, 127)


def groups(x, axis=1):
    """Maxima of groups of 128 columns, [rows, groups]."""
    rows, cols = x.shape
    g = -(-cols // 128)
    p = np.zeros((rows, g * 128))
    p[:, :cols] = np.abs(x)
    return p.reshape(rows, g, 128).max(2)


def fp8_quant(x, fmt):
    """Codes and scale bytes in groups of 128 columns, round-up scales; a group
    with a NaN or an infinity: 0xFF and codes 0x7F."""
    rows, cols = x.shape
    bad = groups(np.where(np.isfinite(x), 0.0, 1.0)) > 0
    clean = np.where(np.isfinite(x), x, 0.0)
    e = ue8m0(groups(clean), fmt)
    full = np.repeat(e, 128, 1)[:, :cols]
    c = nearest(FP8[fmt], np.abs(clean) / np.exp2(full.astype(np.float64))) | (np.signbit(clean) * 0x80)
    badf = np.repeat(bad, 128, 1)[:, :cols]
    return np.where(badf, 0x7F, c).astype(np.uint8), np.where(bad, 0xFF, e + 127).astype(np.uint8)


def fp8_values(codes, scales, fmt):
    t = FP8[fmt]
    m = codes & 0x7F
    v = np.where(m < len(t), t[np.minimum(m, len(t) - 1)], np.nan) * np.where(codes & 0x80, -1.0, 1.0)
    s = np.where(scales == 0xFF, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, 128, 1)[:, :codes.shape[1]]


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_grads(g, u, dh):
    s = sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s
