"""Layer norm and low-rank adapters in 64 bits, and how far the kernels may be
from it.

Roundings are off by at most half a step: U = 2^-24 relative in FP32, 2^-8 in
BF16 (torch.finfo(t).eps / 2).
"""
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def norm(x, w, b, eps):
    """mean, rstd, y and how far y in FP32 may be off.  A row's sum passes at most
    40 additions on the way from one value to the result (8 in a thread, 5 between
    lanes, 16 between warps, some of them for longer rows), so the mean is off by
    D = 40 U mean|x|, a difference by D more than its own rounding, var by 2 D / std
    relatively, rstd by half of that and its own roundings."""
    x = x.double()
    n = x.shape[1]
    mean = x.sum(1, keepdim=True) / n
    rstd = (((x - mean) ** 2).sum(1, keepdim=True) / n + eps).rsqrt()
    w = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(n, dtype=torch.float64, device=x.device) if b is None else b.double()
    xh = (x - mean) * rstd
    d = 40 * U * x.abs().mean(1, keepdim=True) * rstd
    tol = w.abs() * (d + xh.abs() * (d + 40 * U)) + 2 * U * (b.abs() + (xh * w).abs())
    return mean, rstd, xh * w + b, tol


def norm_bwd(dy, x, w, stats, add):
    """dx, dw, db from the stats that the call was given, and their tolerances:
    each of the sums is off by 40 U (rows: rows / 64 + 60, the longest way through
    a CTA's rows and the CTAs' sums) of its values' magnitudes."""
    dy, x = dy.double(), x.double()
    rows, n = x.shape
    mean, rstd = stats.double().split(1, 1)
    w = torch.ones(n, dtype=torch.float64, device=x.device) if w is None else w.double()
    xh = (x - mean) * rstd
    exh = 4 * U * (xh.abs() + (x.abs() + mean.abs()) * rstd * 0.25)
    g = dy * w
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2)
    e1 = 44 * U * g.abs().mean(1, keepdim=True)
    e2 = 44 * U * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * exh).mean(1, keepdim=True)
    tol = rstd * (e1 + xh.abs() * e2 + exh * m2.abs() + 4 * U * (g.abs() + m1.abs() + (xh * m2).abs()))
    if add is not None:
        dx = dx + add.double()
        tol = tol + 2 * U * (add.double().abs() + dx.abs())
    steps = (rows / 64 + 60) * U
    dw, db = (dy * xh).sum(0), dy.sum(0)
    return (dx, tol), (dw, steps * (dy * xh).abs().sum(0) + (dy.abs() * exh).sum(0)), (db, steps * dy.abs().sum(0))


def fp8_groups(y, tol, group, fmt):
    """Values of y as FP8 groups allow them: exponents [rows, groups] of the scales,
    whether tol may move one (y next to a border), and y's own tolerance with the
    code's half step."""
    top, emax = (448.0, 8) if fmt == 0 else (57344.0, 15)
    mant, emin = (3, -6) if fmt == 0 else (2, -14)
    rows, n = y.shape
    width = group or n
    pad = -n % width
    b = torch.nn.functional.pad(y.abs(), (0, pad)).view(rows, -1, width)
    t = torch.nn.functional.pad(tol, (0, pad)).view(rows, -1, width)
    amax, slack = b.amax(2), t.amax(2)

    def exponent(a):
        need = a / top
        m, e = torch.frexp(need)
        e = torch.where(m > 0.5, e, e - 1)            # smallest e with need <= 2^e
        return torch.where(a > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    e = exponent(amax)
    moved = exponent((amax - slack).clamp(min=0)) != exponent(amax + slack)
    scale = torch.exp2(e.double()).repeat_interleave(width, 1)[:, :n]
    v = y / scale
    step = torch.exp2((torch.frexp(v.abs().clamp(min=2.0 ** -100))[1] - 1).double().clamp(min=emin) - mant)
    # a moved scale is twice as coarse
    return e, moved, tol * 1.01 + step * scale * torch.where(moved.repeat_interleave(width, 1)[:, :n], 1.0, 0.5)


def lora(x, a, b, scale, ranks, ids):
    """v, the adapters' addition to y, and its magnitude."""
    t, g = x.shape[0], a.shape[0]
    n, r = b.shape[1], b.shape[2]
    f = dict(dtype=torch.float64, device=x.device)
    v, y, mag, vmag = torch.zeros(t, r, **f), torch.zeros(t, n, **f), torch.zeros(t, n, **f), torch.zeros(t, r, **f)
    for i in range(g):
        rows = (ids == i).nonzero().squeeze(1)
        m = r if ranks is None else max(0, min(r, int(ranks[i])))
        s = 1.0 if scale is None else float(scale[i])
        xa, aa, ba = x[rows].double(), a[i, :m].double(), b[i, :, :m].double()
        v[rows, :m] = xa @ aa.t()
        vmag[rows, :m] = xa.abs() @ aa.abs().t()
        y[rows] = s * (v[rows, :m] @ ba.t())
        mag[rows] = abs(s) * (vmag[rows, :m] @ ba.abs().t())
    return v, vmag, y, mag


def lora_bwd(dy, x, v, a, b, scale, ranks, ids):
    """The additions to dx, dA and dB with their magnitudes."""
    g, r, k = a.shape
    n = b.shape[1]
    f = dict(dtype=torch.float64, device=x.device)
    dx, dxm = torch.zeros(x.shape[0], k, **f), torch.zeros(x.shape[0], k, **f)
    da, dam = torch.zeros(g, r, k, **f), torch.zeros(g, r, k, **f)
    db, dbm = torch.zeros(g, n, r, **f), torch.zeros(g, n, r, **f)
    for i in range(g):
        rows = (ids == i).nonzero().squeeze(1)
        m = r if ranks is None else max(0, min(r, int(ranks[i])))
        s = 1.0 if scale is None else float(scale[i])
        xa, aa, ba, d, va = x[rows].double(), a[i, :m].double(), b[i, :, :m].double(), dy[rows].double(), v[rows, :m].double()
        dv, dvm = s * (d @ ba), abs(s) * (d.abs() @ ba.abs())
        dx[rows], dxm[rows] = dv @ aa, dvm @ aa.abs()
        da[i, :m], dam[i, :m] = dv.t() @ xa, dvm.t() @ xa.abs()
        db[i, :, :m], dbm[i, :, :m] = s * (d.t() @ va), abs(s) * (d.abs().t() @ va.abs())
    return (dx, dxm), (da, dam), (db, dbm)


# How far the adapters' results may be off, of the sum of their products'
# magnitudes.  The tensor core cuts every product of a sum of 16 at 2^-23 of the
# largest term, so a chain of up to 48 such sums (and their two or three parts, whose
# later ones are 2^-8 and 2^-16 of the first) is off by less than 70 * 2^-23; the
# additions to registers add one U each (at most 300 of them here) and a factor in
# two parts 2^-17.  Twice (two products after one another) and rounded up:
MMA = 2 * (70 * 2.0 ** -23 + 300 * U + 2.0 ** -17)


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i].item()!r} for "
                             f"{want[i].item()!r}, tolerance {tol[i].item() if torch.is_tensor(tol) else tol!r}")
