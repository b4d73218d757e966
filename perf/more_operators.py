"""Cases for measuring the layer norm and the low-rank adapters.

What stands before a quantized projection and what is trained beside a frozen
one.  Every case runs in two forms on the same inputs: the plain one (`own`
false), elementary torch operations in 32 bits, and the framework's own kernels
(`own` true), through its public Python functions.  The operators:

  norm       y = (x - mean) rstd w + b in BF16, and / or as the FP8 operand of the
             next product (one scale per token or per 128 columns); mean and rstd
  norm_bwd   gradients of x (added to the residual's gradient), w and b
  lora       y = base + s_g (x A_g^T) B_g^T, g the adapter of the token's request
             (none if negative); x A_g^T kept for the backward pass in training
  lora_bwd   gradients of x (added to the base projection's), A and B

Layer sizes are those of the 1.5B (hidden 1536, MLP 8960) and 7B (hidden 3584,
MLP 18944) layers that the benchmark of this repository runs.
"""
import math

import torch

own = False

EPS = 1e-5


def listed():
    return [
        # decoding: the norm before a 7B layer's projections, one token
        dict(name="norm_1x3584", op="norm", rows=1, cols=3584, pad=0, x="bf16", out="y"),
        # a training step of the 7B layer: the projections' FP8 operand
        dict(name="norm_fp8_token_16384x3584", op="norm", rows=16384, cols=3584, pad=0, x="bf16", out="token"),
        # a short prompt of the 1.5B layer: the FP8 operand per 128 columns, and the rows that adapters read
        dict(name="norm_fp8_group_1000x1536", op="norm", rows=1000, cols=1536, pad=0, x="bf16", out="group+y"),
        # a residual stream in 32 bits, a slice of a wider buffer, sizes that fill nothing
        dict(name="norm_f32_1111x1003", op="norm", rows=1111, cols=1003, pad=37, x="f32", out="y"),
        # the backward of the 7B layer's training step
        dict(name="norm_bwd_16384x3584", op="norm_bwd", rows=16384, cols=3584, x="bf16", add=True),
        # the residual stream in 32 bits, odd rows
        dict(name="norm_bwd_f32_1500x5001", op="norm_bwd", rows=1500, cols=5001, x="f32", add=False),
        # decoding: one token, the 7B layer's gate projection
        dict(name="lora_1x18944x3584", op="lora", t=1, n=18944, k=3584, r=16, g=4, keep=False),
        # decoding a batch of requests with two dozen adapters of different ranks, 1.5B up projection
        dict(name="lora_48x8960x1536", op="lora", t=48, n=8960, k=1536, r=64, g=24, keep=False),
        # several prompts of a few adapters, 7B down projection
        dict(name="lora_4001x3584x18944", op="lora", t=4001, n=3584, k=18944, r=32, g=4, keep=False),
        # fine-tuning one adapter: the forward of the 7B gate projection
        dict(name="lora_8192x18944x3584", op="lora", t=8192, n=18944, k=3584, r=16, g=1, keep=True),
        # and the backward of the 1.5B gate projection, a large adapter
        dict(name="lora_bwd_8192x8960x1536", op="lora_bwd", t=8192, n=8960, k=1536, r=64, g=1),
        # a batch of five users' adapters, sizes that fill no tile
        dict(name="lora_bwd_1000x2050x1999", op="lora_bwd", t=1000, n=2050, k=1999, r=24, g=5),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "lora", "lora", "lora_bwd"])
    if op in ("norm", "norm_bwd"):
        cols = rng.choice([1536, 2048, 3584]) if rng.random() < 0.4 else _spread(rng, 100, 10000)
        rows = _spread(rng, 1 if op == "norm" else 64, min(16384, 16384 * 3584 // cols))
        x = rng.choice(["bf16", "bf16", "f32"])
        if x == "f32":
            rows = (rows + 1) // 2
        if op == "norm_bwd":
            return dict(op=op, rows=rows, cols=cols, x=x, add=rng.random() < 0.5)
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 8, 37]), x=x,
                    out=rng.choice(["y", "y", "token", "group", "token+y", "group+y"]))
    size = lambda: rng.choice([1536, 2048, 3584, 8960]) if rng.random() < 0.5 else _spread(rng, 500, 9000)  # noqa: E731
    r = rng.choice([8, 16, 16, 32, 64]) if rng.random() < 0.7 else rng.randint(1, 64)
    t = _spread(rng, 1 if op == "lora" else 64, 8192)
    g = _spread(rng, 1, min(32 if t <= 256 else 8, t))
    if op == "lora":
        return dict(op=op, t=t, n=size(), k=size(), r=r, g=g, keep=rng.random() < 0.4)
    return dict(op=op, t=t, n=size(), k=size(), r=r, g=g)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _act(g, rows, cols):
    """Activations: channels of different ranges and a few strong outliers."""
    x = _randn(g, rows, cols)
    x *= torch.exp(0.7 * _randn(g, 1, cols))
    x *= torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 1e-3, 30.0, 1.0)
    return x


def _grad(g, rows, cols):
    """Gradients: small, with heavy tails (Student's t, three degrees of freedom)."""
    c = torch.zeros(rows, cols, device="cuda")
    for _ in range(3):
        c += _randn(g, rows, cols).square_()
    return 1e-3 * _randn(g, rows, cols) / (c / 3).sqrt()


def _typed(x, name):
    return x if name == "f32" else x.bfloat16()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, pad = case["rows"], case["cols"], case.get("pad", 0)
        x = _act(g, rows, cols + pad) + 0.3 * _randn(g, rows, 1)
        s["x"] = _typed(x, case["x"])[:, pad:]
        s["weight"], s["bias"] = 1 + 0.2 * _randn(g, cols), 0.1 * _randn(g, cols)
        if op == "norm_bwd":
            # what the forward pass kept
            x = s["x"].float()
            mean = x.mean(1)
            s["stats"] = torch.stack([mean, 1 / (x.var(1, unbiased=False) + EPS).sqrt()], 1)
            s["dy"] = _grad(g, rows, cols).bfloat16()
            s["add"] = _typed(_grad(g, rows, cols), case["x"]) if case["add"] else None
        return s
    t, n, k, r, num = case["t"], case["n"], case["k"], case["r"], case["g"]
    s["a"] = (_randn(g, num, r, k) / math.sqrt(k)).bfloat16()
    s["b"] = (0.05 * _randn(g, num, n, r)).bfloat16()
    s["scale"] = torch.exp(0.5 * _randn(g, num))
    # one adapter is trained at its full rank; those of many users have ranks of their own
    s["ranks"] = torch.full((num,), r, dtype=torch.int32, device="cuda")
    if num > 1:
        s["ranks"][1:] = torch.randint(max(1, r // 4), r + 1, (num - 1,), generator=g, device="cuda").int()
    # requests of one after another's tokens; a few of them without an adapter
    u = torch.rand(t, generator=g, device="cuda")
    ids = (torch.rand(t, generator=g, device="cuda") * num).int().clamp(max=num - 1)
    if t > 256:
        ids = ids[torch.arange(t, device="cuda") // 100 * 100]
        u = u[torch.arange(t, device="cuda") // 100 * 100]
    s["ids"] = torch.where(u < 0.1, -1, ids).int() if num > 1 else torch.zeros_like(ids)
    s["x"] = _act(g, t, k).bfloat16()
    if op == "lora":
        s["base"] = _randn(g, t, n).bfloat16()
    else:
        s["dy"] = _grad(g, t, n).bfloat16()
        s["dx"] = _grad(g, t, k).bfloat16()          # the base projection's
        a = torch.where(_used(s).unsqueeze(2), s["a"], 0).float()
        v = (s["x"].float() @ a.reshape(num * r, k).t()) * _chosen(s)
        s["v"] = v.view(t, num, r).sum(1)            # kept by the forward pass
    if own:
        # the tokens of a batch grouped by adapter: made once, used by every projection of every layer
        import fp8_hybrid_granularity_gb300 as hg
        s["plan"] = hg.lora_plan(s["ids"], num)
    return s


# ---------------------------------------------------------------- plain forms
def _fp8_out(y, group):
    """E4M3 codes and the scales' bytes: the smallest power of two that keeps a
    group (a row for group = 0) within the format."""
    rows, cols = y.shape
    n = group or cols
    b = torch.nn.functional.pad(y, (0, -cols % n)).view(rows, -1, n)
    m, e = torch.frexp(b.abs().amax(2))
    e = e - 9 + (m > 0.875).int()
    e = torch.where(m > 0, e.clamp(-127, 127), torch.full_like(e, -127))
    q = torch.ldexp(b, -e.unsqueeze(2)).view(rows, -1)[:, :cols]
    return q.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _used(s):
    """[g, r]: the rows of A (columns of B) that an adapter of its rank has."""
    return torch.arange(s["r"], device="cuda") < s["ranks"].unsqueeze(1)


def _chosen(s):
    """[t, g r]: 1 where a token's adapter has this row, 0 elsewhere."""
    g = torch.arange(s["g"], device="cuda")
    return ((s["ids"].unsqueeze(1) == g).unsqueeze(2) & _used(s)).flatten(1).float()


def _plain(s):
    op = s["op"]
    if op == "norm":
        x = s["x"].float()
        d = x - x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        y = d * rstd * s["weight"] + s["bias"]
        out = [torch.cat([x.mean(1, keepdim=True), rstd], 1)]
        if "y" in s["out"]:
            out.append(y.bfloat16())
        if s["out"] != "y":
            out += _fp8_out(y, 0 if "token" in s["out"] else 128)
        return out
    if op == "norm_bwd":
        mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
        xh = (s["x"].float() - mean) * rstd
        dy = s["dy"].float()
        g = dy * s["weight"]
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if s["add"] is not None:
            dx = dx + s["add"].float()
        return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    # all adapters' rows side by side; a token takes part in its own adapter's
    num, r, k, n, t = s["g"], s["r"], s["k"], s["n"], s["t"]
    a = s["a"].float().reshape(num * r, k)
    b = s["b"].float().permute(1, 0, 2).reshape(n, num * r)
    chosen = _chosen(s)
    scaled = chosen * s["scale"].repeat_interleave(r)
    if op == "lora":
        v = s["x"].float() @ a.t()
        y = (s["base"].float() + (v * scaled) @ b.t()).bfloat16()
        return (y, (v * chosen).view(t, num, r).sum(1)) if s["keep"] else y
    x, dy = s["x"].float(), s["dy"].float()
    dv = (dy @ b) * scaled
    dx = (s["dx"].float() + dv @ a).bfloat16()
    db = dy.t() @ (s["v"].repeat(1, num) * scaled)
    return dx, (dv.t() @ x).view(num, r, k), db.view(n, num, r).permute(1, 0, 2)


# ---------------------------------------------------------------- the framework's operators
def _shown(q):
    """An FP8 tensor's codes and scale bytes as the numbers they are."""
    return [q.codes.view(torch.float8_e4m3fn), q.scales().view(torch.float8_e8m0fnu)]


def _framework(s):
    import fp8_hybrid_granularity_gb300 as hg
    op = s["op"]
    if op == "norm":
        if s["out"] == "y":
            y, stats = hg.layernorm(s["x"], s["weight"], s["bias"], EPS, out_dtype=torch.bfloat16)
            return [stats, y]
        q, y, stats = hg.fp8_layernorm(s["x"], s["weight"], s["bias"], EPS, group=0 if "token" in s["out"] else 128, with_y="y" in s["out"])
        return [stats] + ([] if y is None else [y]) + _shown(q)
    if op == "norm_bwd":
        return hg.layernorm_bwd(s["dy"], s["x"], s["weight"], s["stats"], add=s["add"])
    adapters = hg.LoraAdapters(s["a"], s["b"], s["scale"], s["ranks"])
    if op == "lora":
        y, v = hg.lora_add(s["base"], s["x"], adapters, s["plan"], keep=s["keep"])
        return (y, v) if s["keep"] else y
    return hg.lora_add_bwd(s["dy"], s["x"], s["v"], adapters, s["plan"], base=s["dx"])


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols = case["rows"], case["cols"]
        n, e = rows * cols, 4 if case["x"] == "f32" else 2
        if op == "norm":
            out = (2 * n if "y" in case["out"] else 0)
            if case["out"] != "y":
                out += n + rows * (1 if "token" in case["out"] else -(-cols // 128))
            return {"bytes": e * n + out + 8 * (rows + cols), "flops": 0}
        return {"bytes": e * n + 2 * n + e * n + (e * n if case["add"] else 0) + 8 * rows + 12 * cols, "flops": 0}
    t, n, k, r = case["t"], case["n"], case["k"], case["r"]
    g = min(case["g"], t)
    if op == "lora":
        return {"bytes": 2 * t * k + 4 * t * n + 2 * g * r * (n + k) + (4 * t * r if case["keep"] else 0), "flops": 2 * t * r * (n + k)}
    return {"bytes": 2 * t * n + 6 * t * k + 4 * t * r + 6 * g * r * (n + k), "flops": 4 * t * r * (n + k)}


# ---------------------------------------------------------------- in 64 bits, from the definitions
def _fp8_64(y, width):
    """Values of the codes, and of the scales, of `width` columns each."""
    codes, scales = torch.zeros_like(y), []
    for j in range(0, y.shape[1], width):
        part = y[:, j:j + width]
        need = part.abs().amax(1, keepdim=True) / 448
        e = torch.frexp(need)[1].double() - 1          # 2^e <= need < 2^(e+1)
        e = torch.where(need > 0, (e + (need > torch.exp2(e))).clamp(-127, 127), torch.full_like(e, -127))
        v = part / torch.exp2(e)
        step = torch.exp2((torch.frexp(v.abs().clamp(min=2.0 ** -100))[1] - 1).double().clamp(min=-6)) / 8
        codes[:, j:j + width] = torch.round(v / step) * step
        scales.append(torch.exp2(e))
    return [codes, torch.cat(scales, 1)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
        y = (x - mean) / (var + EPS).sqrt() * w + b
        out = [torch.cat([mean, (var + EPS).rsqrt()], 1)] + ([y] if "y" in case["out"] else [])
        if case["out"] != "y":
            out += _fp8_64(y, case["cols"] if "token" in case["out"] else 128)
        return out
    if op == "norm_bwd":
        mean, rstd = s["stats"].double().split(1, 1)
        dy, n = s["dy"].double(), case["cols"]
        xh = (s["x"].double() - mean) * rstd
        g = dy * s["weight"].double()
        dx = rstd * (g - g.sum(1, keepdim=True) / n - xh * (g * xh).sum(1, keepdim=True) / n)
        return dx if s["add"] is None else dx + s["add"].double(), torch.einsum("ij,ij->j", dy, xh), dy.sum(0)
    t, n, k, r = case["t"], case["n"], case["k"], case["r"]
    x = s["x"].double()
    if op == "lora":
        y, v = s["base"].double(), torch.zeros(t, r, dtype=torch.float64, device="cuda")
    else:
        dy, v, dx = s["dy"].double(), s["v"].double(), s["dx"].double()
        da = torch.zeros(case["g"], r, k, dtype=torch.float64, device="cuda")
        db = torch.zeros(case["g"], n, r, dtype=torch.float64, device="cuda")
    for i in range(case["g"]):
        rows = (s["ids"] == i).nonzero().squeeze(1)
        m, f = int(s["ranks"][i]), float(s["scale"][i])
        a, b = s["a"][i, :m].double(), s["b"][i, :, :m].double()
        if op == "lora":
            v[rows, :m] = x[rows] @ a.t()
            y[rows] += f * (v[rows, :m] @ b.t())
        else:
            dv = f * (dy[rows] @ b)
            dx[rows] += dv @ a
            da[i, :m] = dv.t() @ x[rows]
            db[i, :, :m] = f * (dy[rows].t() @ v[rows, :m])
    if op == "lora":
        return (y, v) if case["keep"] else y
    return dx, da, db
