"""Low-rank adapters beside a projection, forward and backward, against 64 bits."""
import pytest
import torch

import adapt_ref as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
# tokens, n, k, r, adapters
SIZES = [(1, 64, 64, 16, 1), (1, 130, 70, 5, 3), (5, 8, 8, 1, 1), (7, 257, 129, 8, 4), (33, 1536, 264, 64, 12),
         (129, 384, 640, 16, 2), (300, 1003, 517, 24, 5), (513, 256, 2048, 64, 7), (260, 300, 333, 128, 2),
         (1000, 264, 200, 100, 3), (128, 128, 128, 32, 1), (2000, 512, 320, 16, 1), (64, 72, 4096, 32, 64)]


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda"))


def batch(t, n, k, r, g, seed=0, none=0.15):
    gen = torch.Generator().manual_seed(seed + t * 7 + n)
    ids = torch.randint(0, g, (t,), generator=gen, dtype=torch.int32)
    ids[torch.rand(t, generator=gen) < none] = -1
    ranks = torch.randint(max(1, r // 3), r + 1, (g,), generator=gen, dtype=torch.int32)
    ranks[0] = r
    a, b = rand(seed + 1, g, r, k, scale=k ** -0.5).bfloat16(), rand(seed + 2, g, n, r, scale=0.3).bfloat16()
    return dict(x=rand(seed + 3, t, k).bfloat16(), dy=rand(seed + 4, t, n).bfloat16(), a=a, b=b,
                scale=torch.exp(rand(seed + 5, g)), ranks=ranks.cuda(), ids=ids.cuda())


def adapters(lib, s):
    return lib.LoraAdapters(s["a"], s["b"], s["scale"], s["ranks"])


def check_forward(s, base, y, v=None):
    want_v, vmag, add, mag = ref.lora(s["x"], s["a"], s["b"], s["scale"], s["ranks"], s["ids"])
    want = add if base is None else base.double() + add
    ref.close(y, want, ref.MMA * mag + (ref.half_step(y.dtype) + 2 * ref.U) * 1.01 * want.abs(), "y")
    if v is not None:
        ref.close(v, want_v, ref.MMA * vmag, "v")
    return want_v


def check_backward(s, base, v, dx, da, db):
    (wx, mx), (wa, ma), (wb, mb) = ref.lora_bwd(s["dy"], s["x"], v, s["a"], s["b"], s["scale"], s["ranks"], s["ids"])
    wx = wx if base is None else wx + base.double()
    ref.close(dx, wx, ref.MMA * mx + (ref.half_step(dx.dtype) + 2 * ref.U) * 1.01 * wx.abs(), "dx")
    if da is not None:
        ref.close(da, wa, ref.MMA * ma + ref.half_step(da.dtype) * 1.01 * wa.abs(), "dA")
        ref.close(db, wb, ref.MMA * mb + ref.half_step(db.dtype) * 1.01 * wb.abs(), "dB")
    return wx, wa, wb


@pytest.mark.parametrize("t,g", [(0, 1), (1, 1), (31, 2), (1000, 7), (5000, 300), (777, 4096), (70000, 3), (129, 1)])
def test_plan(cuda_lib, t, g):
    gen = torch.Generator().manual_seed(t + g)
    ids = torch.randint(-1, g + 1, (t,), generator=gen, dtype=torch.int32)     # g: one too many, without an adapter
    p = cuda_lib.lora_plan(ids.cuda(), g)
    w = p.words.cpu()
    bucket = torch.where((ids >= 0) & (ids < g), ids, g)
    counts = torch.bincount(bucket.long(), minlength=g + 1)
    starts = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    assert torch.equal(w[4:4 + g + 2].long(), starts)
    tiles = -(-counts // 128)
    first = torch.cat([torch.zeros(1, dtype=torch.long), tiles.cumsum(0)])
    assert torch.equal(w[6 + g:8 + 2 * g].long(), first) and int(w[0]) == int(first[-1])
    at = 8 + 2 * g
    assert torch.equal(w[at:at + t].long(), torch.sort(bucket, stable=True)[1])
    at += t + -(at + t) % 4
    got = w[at:at + 4 * int(w[0])].view(-1, 4)
    want = [(i if i < g else -1, int(starts[i]) + 128 * j, min(128, int(counts[i]) - 128 * j)) for i in range(g + 1) for j in range(int(tiles[i]))]
    assert got[:, :3].tolist() == [list(e) for e in want]
    for _, first, count, row in got.tolist():
        tokens = w[8 + 2 * g + first:8 + 2 * g + first + count].tolist()
        assert row == (tokens[0] if tokens == list(range(tokens[0], tokens[0] + count)) else -1)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_forward(cuda_lib, size, dtype):
    t, n = size[:2]
    s = batch(*size)
    plan = cuda_lib.lora_plan(s["ids"], size[4])
    base = rand(9, t, n).to(dtype)
    y, v = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, keep=True)
    check_forward(s, base, y, v)
    none = s["ids"] < 0
    assert torch.equal(y[none], base[none]) and (v[none] == 0).all()
    again, _ = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan)
    assert torch.equal(again, y)
    z, _ = cuda_lib.lora_add(None, s["x"], adapters(cuda_lib, s), plan, out_dtype=dtype)
    check_forward(s, None, z)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype,grads", [(BF16, F32), (F32, BF16)])
def test_backward(cuda_lib, size, dtype, grads):
    t, n, k, r, g = size
    s = batch(*size)
    plan = cuda_lib.lora_plan(s["ids"], g)
    v = ref.lora(s["x"], s["a"], s["b"], s["scale"], s["ranks"], s["ids"])[0].float()
    base = rand(8, t, k).to(dtype)
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan, base=base, params_dtype=grads)
    assert dx.dtype == dtype and da.dtype == db.dtype == grads
    _, wa, wb = check_backward(s, base, v, dx, da, db)
    if grads == F32:
        # not only every value within its bound: the whole within FP32's
        for got, want in ((da, wa), (db, wb)):
            assert float((got.double() - want).norm()) <= 4e-6 * float(want.norm())
    only, none, _ = cuda_lib.lora_add_bwd(s["dy"], None, None, adapters(cuda_lib, s), plan, base=base, params=False)
    assert torch.equal(only, dx) and none is None
    z, _, _ = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan, out_dtype=dtype)
    check_backward(s, None, v, z, None, None)


@pytest.mark.parametrize("t,g,none", [(1000, 4, 0.6), (4001, 4, 0.12), (700, 2, 0.97), (130, 1, 0.0)])
def test_long_sides(cuda_lib, t, g, none):
    """Many steps of the long sides, with fewer tiles than the tokens would fill."""
    n, k, r = 1104, 4096, 32
    s = batch(t, n, k, r, g, none=none)
    plan = cuda_lib.lora_plan(s["ids"], g)
    base = rand(9, t, n).bfloat16()
    y, v = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, keep=True)
    check_forward(s, base, y, v)
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan)
    check_backward(s, None, v, dx, da, db)


def test_past_the_rank_and_without_an_adapter(cuda_lib):
    """What lies past a rank, and the rows of tokens without an adapter, may be
    anything; an adapter of rank 0 adds nothing."""
    s = batch(200, 264, 136, 24, 4)
    s["ranks"] = torch.tensor([24, 0, 5, 17], dtype=torch.int32, device="cuda")
    nan = float("nan")
    for i, m in enumerate(s["ranks"].tolist()):
        s["a"][i, m:], s["b"][i, :, m:] = nan, nan
    none = s["ids"] < 0
    assert none.any()
    clean = {**s, "x": s["x"].clone(), "dy": s["dy"].clone()}
    s["x"][none], s["dy"][none] = nan, float("inf")
    plan = cuda_lib.lora_plan(s["ids"], 4)
    base = rand(9, 200, 264).bfloat16()
    y, v = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, keep=True)
    want_v = check_forward(clean, base, y, v)
    v2 = want_v.float()
    v2[none] = nan
    for i, m in enumerate(s["ranks"].tolist()):
        rows = (s["ids"] == i).nonzero()
        v2[rows, torch.arange(m, 24, device="cuda")] = nan
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v2, adapters(cuda_lib, s), plan)
    check_backward(clean, None, want_v, dx, da, db)
    assert (da[1] == 0).all() and (db[1] == 0).all() and (da[2, 5:] == 0).all() and (db[3, :, 17:] == 0).all()


def test_non_finite_tokens_stay_their_own(cuda_lib):
    """A token with a NaN or an infinity spoils its own row and its own adapter's
    gradients, not its neighbours'."""
    s = batch(150, 264, 136, 16, 2, none=0.0)
    i = int((s["ids"] == 0).nonzero()[3])
    s["x"][i, 7] = float("inf")
    s["dy"][i, 9] = float("nan")
    plan = cuda_lib.lora_plan(s["ids"], 2)
    y, v = cuda_lib.lora_add(None, s["x"], adapters(cuda_lib, s), plan, keep=True)
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan)
    others = torch.arange(150, device="cuda") != i
    assert y[others].isfinite().all() and dx[others].isfinite().all() and not y[i].isfinite().any()
    assert da[1].isfinite().all() and db[1].isfinite().all() and not da[0].isfinite().any()


@pytest.mark.parametrize("pad", [1, 2, 8])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(cuda_lib, pad, dtype):
    t, n, k, r, g = 140, 200, 168, 16, 3
    s = batch(t, n, k, r, g)
    wide = lambda x: torch.nn.functional.pad(x, (pad, pad), value=float("nan"))[..., pad:pad + x.shape[-1]]  # noqa: E731
    w = {**s, "x": wide(s["x"]), "dy": wide(s["dy"]), "a": wide(s["a"]), "b": wide(s["b"])}
    plan = cuda_lib.lora_plan(s["ids"], g)
    base, whole = wide(rand(9, t, n).to(dtype)), torch.full((t, n + 2 * pad), 7.0, dtype=dtype, device="cuda")
    y, v = cuda_lib.lora_add(base, w["x"], adapters(cuda_lib, w), plan, out=whole[:, pad:pad + n], keep=True)
    check_forward(s, base, y, v)
    whole[:, pad:pad + n] = 7.0
    assert (whole == 7.0).all()
    dbase, whole = wide(rand(8, t, k).to(dtype)), torch.full((t, k + 2 * pad), 7.0, dtype=dtype, device="cuda")
    dx, da, db = cuda_lib.lora_add_bwd(w["dy"], w["x"], wide(v), adapters(cuda_lib, w), plan, base=dbase, out=whole[:, pad:pad + k])
    check_backward(s, dbase, v, dx, da, db)
    whole[:, pad:pad + k] = 7.0
    assert (whole == 7.0).all()


# tokens, n, k, r, adapters: up to 16 tokens, up to 64 with many adapters, several 16s of
# one, a long side past the one-kernel form's
@pytest.mark.parametrize("size", [(1, 260, 72, 8, 1), (1, 4, 8, 16, 3), (2, 4100, 520, 128, 2), (5, 36, 8, 40, 2), (16, 132, 4104, 16, 1),
                                  (17, 1028, 520, 24, 5), (48, 520, 264, 64, 24), (64, 260, 136, 32, 16), (64, 2052, 88, 128, 64),
                                  (33, 68, 1056, 16, 9), (9, 64, 49152, 16, 2), (9, 64, 49160, 16, 2), (20, 96, 64, 8, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_tokens(cuda_lib, size, dtype):
    """Decoding: what lies past a rank, and rows of tokens without an adapter, may be
    anything; rows of wider buffers; y over base."""
    t, n, k, r, g = size
    s = batch(*size, seed=40, none=0.1)
    for i, m in enumerate(s["ranks"].tolist()):
        s["a"][i, m:], s["b"][i, :, m:] = float("nan"), float("nan")
    none = s["ids"] < 0
    s["x"][none] = float("nan")
    wide = lambda x: torch.nn.functional.pad(x, (8, 8), value=float("nan"))[..., 8:8 + x.shape[-1]]  # noqa: E731
    w = {**s, "x": wide(s["x"]), "a": wide(s["a"]), "b": wide(s["b"])}
    plan = cuda_lib.lora_plan(s["ids"], g)
    base, whole = wide(rand(9, t, n).to(dtype)), torch.full((t, n + 16), 7.0, dtype=dtype, device="cuda")
    y, v = cuda_lib.lora_add(base, w["x"], adapters(cuda_lib, w), plan, out=whole[:, 8:8 + n], keep=True)
    s["x"][none] = 0.0
    check_forward(s, base, y, v)
    assert torch.equal(y[none], base[none]) and (v[none] == 0).all()
    z, _ = cuda_lib.lora_add(None, w["x"], adapters(cuda_lib, w), plan, out_dtype=dtype)
    check_forward(s, None, z)
    y = y.clone()
    assert torch.equal(cuda_lib.lora_add(base, w["x"], adapters(cuda_lib, w), plan, out=base)[0], y)
    whole[:, 8:8 + n] = 7.0
    assert (whole == 7.0).all()


def test_in_place_defaults_and_empty(cuda_lib):
    t, n, k, r, g = 100, 256, 128, 16, 2
    s = batch(t, n, k, r, g)
    s["scale"], s["ranks"] = None, None
    plan = cuda_lib.lora_plan(s["ids"], g)
    base = rand(9, t, n).bfloat16()
    want, v = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, keep=True)
    check_forward(s, base, want, v)
    got, _ = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, out=base)
    assert got.data_ptr() == base.data_ptr() and torch.equal(got, want)
    dbase = rand(8, t, k).bfloat16()
    want = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan, base=dbase)
    check_backward(s, dbase, v, *want)
    got = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan, base=dbase, out=dbase)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    # no token at all, and none with an adapter
    for ids in (s["ids"][:0], torch.full((3,), -1, dtype=torch.int32, device="cuda")):
        m = ids.shape[0]
        p = cuda_lib.lora_plan(ids, g)
        b0 = rand(9, m, n).bfloat16()
        y, v0 = cuda_lib.lora_add(b0, s["x"][:m], adapters(cuda_lib, s), p, keep=True)
        assert torch.equal(y, b0) and (v0 == 0).all()
        dx, da, db = cuda_lib.lora_add_bwd(s["dy"][:m], s["x"][:m], v0, adapters(cuda_lib, s), p, base=dbase[:m])
        assert torch.equal(dx, dbase[:m]) and (da == 0).all() and (db == 0).all()


def test_gradients_by_differences(cuda_lib):
    """sum(y * c) is linear in x, A and B one at a time: differences are exact."""
    t, n, k, r, g = 12, 24, 40, 8, 2
    s = batch(t, n, k, r, g)
    plan = cuda_lib.lora_plan(s["ids"], g)
    ad = adapters(cuda_lib, s)
    _, v = cuda_lib.lora_add(None, s["x"], ad, plan, keep=True)
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, ad, plan, out_dtype=F32)

    def f(**change):
        d = {**s, **change}
        return (ref.lora(d["x"], d["a"], d["b"], s["scale"], s["ranks"], s["ids"])[2] * s["dy"].double()).sum()

    for name, got in (("x", dx), ("a", da), ("b", db)):
        for i in range(0, s[name].numel(), max(1, s[name].numel() // 9)):
            up, down = (s[name].double().clone() for _ in range(2))
            up.view(-1)[i] += 1
            down.view(-1)[i] -= 1
            want = float(f(**{name: up}) - f(**{name: down})) / 2
            assert abs(float(got.reshape(-1)[i]) - want) < 1e-4 * (1 + abs(want)), (name, i)


def test_captured(cuda_lib):
    """A graph of plan, forward and backward replays with new tokens and adapters."""
    size = (300, 256, 512, 16, 5)
    s, s2 = batch(*size), batch(*size, seed=50)
    base = rand(9, 300, 256).bfloat16()

    def step(s):
        plan = cuda_lib.lora_plan(s["ids"], 5)
        y, v = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, keep=True)
        return (y, v) + cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan)

    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s)
    for name in s:
        s[name].copy_(s2[name])
    graph.replay()
    want = step(s2)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))


def test_other_stream(cuda_lib):
    size = (300, 256, 512, 16, 5)
    s = batch(*size)
    base = rand(9, 300, 256).bfloat16()
    plan = cuda_lib.lora_plan(s["ids"], 5)
    want, v = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, keep=True)
    grads = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    plan = cuda_lib.lora_plan(s["ids"], 5, stream=st)
    y, v2 = cuda_lib.lora_add(base, s["x"], adapters(cuda_lib, s), plan, keep=True, stream=st)
    got = cuda_lib.lora_add_bwd(s["dy"], s["x"], v2, adapters(cuda_lib, s), plan, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(y, want) and all(torch.equal(p, q) for p, q in zip(got, grads))
