"""Adapters at the edges of what a call may be given: non-finite values beside ranks,
long sides that only the length of sums splits, offsets past 32 bits."""
import pytest
import torch

import adapt_ref as ref
from test_gpu_lora import adapters, batch, check_backward, check_forward, rand

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("t,n,k,r", [(200, 264, 136, 24), (2500, 264, 136, 64), (2500, 137, 131, 128), (40, 264, 136, 16)])
@pytest.mark.parametrize("grads", [F32, BF16])
def test_zeros_past_the_rank_whatever_the_tokens_hold(cuda_lib, t, n, k, r, grads):
    """An infinity or a NaN among an adapter's tokens leaves dA and dB past its rank
    zero, and all of an adapter of rank 0 (sums of one chunk and of several)."""
    s = batch(t, n, k, r, 3)
    s["ranks"] = torch.tensor([0, r // 3, r], dtype=torch.int32, device="cuda")
    plan = cuda_lib.lora_plan(s["ids"], 3)
    _, v = cuda_lib.lora_add(None, s["x"], adapters(cuda_lib, s), plan, keep=True)
    for g in (0, 1):
        rows = (s["ids"] == g).nonzero().squeeze(1)
        s["x"][rows[0], 3], s["x"][rows[-1], 5] = float("inf"), float("nan")
        s["dy"][rows[0], 7], s["dy"][rows[-1], 2] = float("-inf"), float("nan")
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan, params_dtype=grads)
    m = r // 3
    assert (da[0] == 0).all() and (db[0] == 0).all() and (da[1, m:] == 0).all() and (db[1, :, m:] == 0).all()
    # within the rank such gradients are not finite, other adapters' are
    assert not da[1, :m, 3].isfinite().any() and not db[1, 7, :m].isfinite().any()
    assert da[2].isfinite().all() and db[2].isfinite().all()


# tokens, long side, r: more tiles than CTAs, so that only the limit of a sum's length
# splits the long side (two, three splits); few tokens and more splits than CTAs would
# be given (17, 33, 35)
@pytest.mark.parametrize("t,long_side,r", [(19500, 8200, 16), (19500, 8200, 128), (20, 98400, 16), (20, 98400, 128), (70, 106501, 100)])
def test_splits_that_the_length_of_sums_asks_for(cuda_lib, t, long_side, r):
    """Forward over a long k, backward over a long n, some tokens without an adapter."""
    short, g = 64, 3
    sel = torch.arange(0, t, max(1, t // 64), device="cuda")
    part = lambda s, **k: {**s, "x": s["x"][sel], "dy": s["dy"][sel], "ids": s["ids"][sel], **k}  # noqa: E731
    s = batch(t, short, long_side, r, g)
    plan = cuda_lib.lora_plan(s["ids"], g)
    y, v = cuda_lib.lora_add(None, s["x"], adapters(cuda_lib, s), plan, keep=True, out_dtype=F32)
    check_forward(part(s), None, y[sel], v[sel])
    s = batch(t, long_side, short, r, g)
    s["dy"] *= long_side ** -0.5
    plan = cuda_lib.lora_plan(s["ids"], g)
    v = rand(6, t, r)
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, adapters(cuda_lib, s), plan, out_dtype=F32)
    p = part(s)
    (wx, mx), _, _ = ref.lora_bwd(p["dy"], p["x"], v[sel].double(), s["a"], s["b"], s["scale"], s["ranks"], p["ids"])
    ref.close(dx[sel], wx, ref.MMA * mx + 3 * ref.U * wx.abs(), "dx")
    if t * long_side * r < 1 << 32:
        wv = ref.lora_bwd(s["dy"], s["x"], v.double(), s["a"], s["b"], s["scale"], s["ranks"], s["ids"])[1]
        ref.close(da, wv[0], ref.MMA * wv[1] + ref.U * wv[0].abs(), "dA")
    # some of n's columns, the last ones among them
    cols = torch.cat([torch.arange(0, long_side, 997, device="cuda"), torch.arange(long_side - 5, long_side, device="cuda")])
    _, _, (wb, mb) = ref.lora_bwd(s["dy"][:, cols], s["x"], v.double(), s["a"], s["b"][:, cols], s["scale"], s["ranks"], s["ids"])
    ref.close(db[:, cols], wb, ref.MMA * mb + ref.U * wb.abs(), "dB")


@pytest.mark.parametrize("t,kind,at", [(6, BF16, 16), (6, F32, 16), (140, BF16, 16), (140, F32, 16), (140, BF16, 5), (140, F32, 5)])
def test_rows_far_apart(cuda_lib, t, kind, at):
    """Row offsets that pass 2^31 elements: every matrix a slice of a wide buffer."""
    n, k, r, g = 264, 136, 16, 3
    s = batch(t, n, k, r, g)
    width = (1 << 31) // (t - 2) // 16 * 16 + (0 if at == 16 else 3)
    wide = torch.empty(t, width, dtype=BF16, device="cuda")
    wide_f = torch.empty(t, width, dtype=F32, device="cuda") if kind == F32 else wide

    def place(buf, x, i):
        to = buf[:, at + 1024 * i:at + 1024 * i + x.shape[1]]
        return to.copy_(x)
    x, dy = place(wide, s["x"], 0), place(wide, s["dy"], 1)
    base, dbase = place(wide_f, rand(9, t, n).to(kind), 2), place(wide_f, rand(8, t, k).to(kind), 3)
    out, dout = wide_f[:, at + 4096:at + 4096 + n], wide_f[:, at + 5120:at + 5120 + k]
    assert out[-1].data_ptr() - out.data_ptr() >= (1 << 31) * kind.itemsize
    plan = cuda_lib.lora_plan(s["ids"], g)
    w = {**s, "x": x, "dy": dy}
    y, v = cuda_lib.lora_add(base, x, adapters(cuda_lib, s), plan, out=out, keep=True)
    check_forward(w, base, y, v)
    dx, da, db = cuda_lib.lora_add_bwd(dy, x, v, adapters(cuda_lib, s), plan, base=dbase, out=dout)
    check_backward(w, dbase, v, dx, da, db)


def test_adapters_far_apart(cuda_lib):
    """A bank of more than 2^31 elements, its gradients as well; two adapters in use."""
    t, n, k, r, g = 130, 72, 4104, 128, 4096
    s = batch(t, n, k, r, 2, none=0.1)
    a, b = torch.empty(g, r, k, dtype=BF16, device="cuda"), torch.empty(g, n, r, dtype=BF16, device="cuda")
    a[0], a[-1], b[0], b[-1] = s["a"][0], s["a"][1], s["b"][0], s["b"][1]
    scale, ranks = torch.ones(g, device="cuda"), torch.full((g,), r, dtype=torch.int32, device="cuda")
    scale[0], scale[-1], ranks[0], ranks[-1] = s["scale"][0], s["scale"][1], s["ranks"][0], s["ranks"][1]
    assert a.numel() > 1 << 31
    ids = torch.where(s["ids"] == 1, g - 1, s["ids"]).int()
    plan = cuda_lib.lora_plan(ids, g)
    w = cuda_lib.LoraAdapters(a, b, scale, ranks)
    y, v = cuda_lib.lora_add(None, s["x"], w, plan, keep=True)
    check_forward(s, None, y, v)
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, w, plan, params_dtype=BF16)
    check_backward(s, None, v, dx, da[[0, -1]], db[[0, -1]])
    assert not da[1:-1].any() and not db[1:-1].any()


@pytest.mark.parametrize("t,n,k,r,g", [(1 << 24, 64, 64, 16, 4096), (1 << 20, 65, 129, 24, 300), (3, 1 << 24, 64, 8, 2), (200, (1 << 21) + 1, 63, 9, 2),
                                       (3, 64, 1 << 24, 8, 2), (200, 64, 1 << 22, 16, 2)])
def test_largest_sizes(cuda_lib, t, n, k, r, g):
    """As many tokens, adapters and columns as a call takes: some rows of y, v and dx, some
    columns of three adapters' gradients."""
    s = dict(ids=torch.randint(-1, g, (t,), device="cuda", dtype=torch.int32), ranks=torch.randint(1, r + 1, (g,), device="cuda", dtype=torch.int32),
             scale=torch.exp(0.3 * rand(5, g)))
    for name, shape, scale in (("x", (t, k), 1.0), ("dy", (t, n), n ** -0.5), ("a", (g, r, k), k ** -0.5), ("b", (g, n, r), 0.3)):
        s[name] = scale * torch.randn(*shape, device="cuda", dtype=BF16)
    plan = cuda_lib.lora_plan(s["ids"], g)
    w = adapters(cuda_lib, s)
    y, v = cuda_lib.lora_add(None, s["x"], w, plan, keep=True)
    dx, da, db = cuda_lib.lora_add_bwd(s["dy"], s["x"], v, w, plan)
    assert cuda_lib.fp8hg_get_device_error() == 0
    some = lambda size: torch.cat([torch.arange(0, size, max(1, size // 300), device="cuda"),  # noqa: E731
                                   torch.arange(max(0, size - 200), size, device="cuda")]).unique()
    sel, cols, kcols = some(t), some(n), some(k)
    p = {**s, "x": s["x"][sel], "dy": s["dy"][sel], "ids": s["ids"][sel]}
    check_forward(p, None, y[sel], v[sel])
    (wx, mx), _, _ = ref.lora_bwd(p["dy"], p["x"], v[sel].double(), s["a"], s["b"], s["scale"], s["ranks"], p["ids"])
    ref.close(dx[sel], wx, ref.MMA * mx + (ref.half_step(BF16) + 2 * ref.U) * 1.01 * wx.abs(), "dx")
    for i in {0, g // 2, g - 1}:
        rows, m, f = (s["ids"] == i).nonzero().squeeze(1), int(s["ranks"][i]), float(s["scale"][i])
        va, b, d = v[rows, :m].double(), s["b"][i, :, :m].double(), s["dy"][rows].double()
        dv, dvm, x, d = f * (d @ b), f * (d.abs() @ b.abs()), s["x"][rows][:, kcols].double(), d[:, cols]
        for got, want, mag in ((da[i, :m][:, kcols], dv.t() @ x, dvm.t() @ x.abs()), (db[i, cols, :m], f * (d.t() @ va), f * (d.abs().t() @ va.abs()))):
            ref.close(got, want, ref.MMA * mag + ref.U * want.abs(), "dA or dB")
        assert not da[i, m:].any() and not db[i, :, m:].any()
