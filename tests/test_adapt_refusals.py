"""The Python side of the layer norm and adapter calls without a GPU: what is
refused before anything reaches the library.  Tensors on a GPU are stood in for;
no call here launches anything."""
import pytest
import torch

import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import adapt, lowbit
from test_lowbit_refusals import Reached, StandIn

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def gpu0(monkeypatch):
    """GPU 0 is current; the library only says that it was reached."""
    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_workspace") or name.endswith("_bytes"):
                    return 4096
                raise Reached(name)
            return call

    monkeypatch.setattr(lowbit, "_cuda_device", lambda: 0)
    monkeypatch.setattr(lowbit, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(lowbit, "_scratch", lambda n, x, stream: StandIn(torch.empty(n, dtype=torch.uint8)))
    monkeypatch.setattr(adapt, "_fns", Library)
    monkeypatch.setattr(adapt, "_bound", None)
    monkeypatch.setattr(adapt, "_new", lambda *a: StandIn(torch.empty_strided(*a[:2], dtype=a[2])))
    adapt._bytes.cache_clear()
    yield StandIn
    adapt._bytes.cache_clear()


def z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


T, N, K, R, G = 6, 24, 16, 8, 2


def adapters(on, **one):
    f = {"a": z(G, R, K), "b": z(G, N, R), "scale": z(G, dtype=F32), "ranks": z(G, dtype=torch.int32)}
    return fp8hg.LoraAdapters(*(one[n](t) if n in one else on(t) for n, t in f.items()))


def plan(on, tokens=T, g=G):
    return fp8hg.LoraPlan(on(z(64, dtype=torch.int32)), tokens, g)


# every tensor argument of every call: the call with one argument from `one`, the others from `on`
CALLS = {
    "norm x": lambda on, one: fp8hg.layernorm(one(z(4, 8)), on(z(8)), on(z(8))),
    "norm weight": lambda on, one: fp8hg.layernorm(on(z(4, 8)), one(z(8)), on(z(8))),
    "norm bias": lambda on, one: fp8hg.layernorm(on(z(4, 8)), on(z(8)), one(z(8))),
    "norm bias alone": lambda on, one: fp8hg.layernorm(on(z(4, 8)), None, one(z(8))),
    "norm out": lambda on, one: fp8hg.layernorm(on(z(4, 8)), out=one(z(4, 8))),
    "fp8 norm x": lambda on, one: fp8hg.fp8_layernorm(one(z(4, 8)), on(z(8)), on(z(8)), group=128),
    "fp8 norm weight": lambda on, one: fp8hg.fp8_layernorm(on(z(4, 8)), one(z(8)), on(z(8))),
    "bwd dy": lambda on, one: fp8hg.layernorm_bwd(one(z(4, 8)), on(z(4, 8)), on(z(8)), on(z(4, 2, dtype=F32))),
    "bwd x": lambda on, one: fp8hg.layernorm_bwd(on(z(4, 8)), one(z(4, 8)), on(z(8)), on(z(4, 2, dtype=F32))),
    "bwd weight": lambda on, one: fp8hg.layernorm_bwd(on(z(4, 8)), on(z(4, 8)), one(z(8)), on(z(4, 2, dtype=F32))),
    "bwd stats": lambda on, one: fp8hg.layernorm_bwd(on(z(4, 8)), on(z(4, 8)), None, one(z(4, 2, dtype=F32))),
    "bwd add": lambda on, one: fp8hg.layernorm_bwd(on(z(4, 8)), on(z(4, 8)), None, on(z(4, 2, dtype=F32)), add=one(z(4, 8))),
    "bwd out": lambda on, one: fp8hg.layernorm_bwd(on(z(4, 8)), on(z(4, 8)), None, on(z(4, 2, dtype=F32)), out=one(z(4, 8))),
    "plan ids": lambda on, one: fp8hg.lora_plan(one(z(T, dtype=torch.int32)), G),
    "add base": lambda on, one: fp8hg.lora_add(one(z(T, N)), on(z(T, K)), adapters(on), plan(on)),
    "add x": lambda on, one: fp8hg.lora_add(on(z(T, N)), one(z(T, K)), adapters(on), plan(on)),
    "add out": lambda on, one: fp8hg.lora_add(on(z(T, N)), on(z(T, K)), adapters(on), plan(on), out=one(z(T, N))),
    "add plan": lambda on, one: fp8hg.lora_add(None, on(z(T, K)), adapters(on), plan(one)),
    "add_bwd dy": lambda on, one: fp8hg.lora_add_bwd(one(z(T, N)), on(z(T, K)), on(z(T, R, dtype=F32)), adapters(on), plan(on)),
    "add_bwd x": lambda on, one: fp8hg.lora_add_bwd(on(z(T, N)), one(z(T, K)), on(z(T, R, dtype=F32)), adapters(on), plan(on)),
    "add_bwd v": lambda on, one: fp8hg.lora_add_bwd(on(z(T, N)), on(z(T, K)), one(z(T, R, dtype=F32)), adapters(on), plan(on)),
    "add_bwd base": lambda on, one: fp8hg.lora_add_bwd(on(z(T, N)), on(z(T, K)), on(z(T, R, dtype=F32)), adapters(on), plan(on),
                                                       base=one(z(T, K))),
    "add_bwd out": lambda on, one: fp8hg.lora_add_bwd(on(z(T, N)), None, None, adapters(on), plan(on), out=one(z(T, K)), params=False),
    "add_bwd plan": lambda on, one: fp8hg.lora_add_bwd(on(z(T, N)), None, None, adapters(on), plan(one), params=False),
}
for field in ("a", "b", "scale", "ranks"):
    CALLS["adapters " + field] = lambda on, one, field=field: fp8hg.lora_add(None, on(z(T, K)), adapters(on, **{field: one}), plan(on))


@pytest.mark.parametrize("name", CALLS)
def test_tensors_elsewhere_are_refused(gpu0, name):
    """A call launches on the current device: tensors of another GPU, or of the
    CPU, never reach it."""
    with pytest.raises(Reached):
        CALLS[name](gpu0, gpu0)
    for elsewhere in (lambda t: StandIn(t, 1), lambda t: t):
        with pytest.raises(ValueError):
            CALLS[name](gpu0, elsewhere)


def test_types_shapes_and_strides(gpu0):
    on = gpu0
    ok = lambda **k: {**dict(x=on(z(4, 8)), weight=on(z(8)), bias=on(z(8))), **k}  # noqa: E731
    for bad in (dict(x=on(z(4, 8, dtype=torch.float16))), dict(x=on(z(8))), dict(x=on(z(8, 4).t())), dict(weight=on(z(9))),
                dict(weight=on(z(16)[::2])), dict(weight=on(z(8, dtype=F32))), dict(bias=on(z(8, dtype=torch.float16))),
                dict(out=on(z(4, 9))), dict(out=on(z(8, 4).t())), dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            fp8hg.layernorm(**ok(**bad))
            pytest.fail(str(bad.keys()))
    with pytest.raises(ValueError):
        fp8hg.fp8_layernorm(on(z(4, 8)), group=64)
    stats = on(z(4, 2, dtype=F32))
    ok = lambda **k: {**dict(dy=on(z(4, 8)), x=on(z(4, 8)), weight=None, stats=stats), **k}  # noqa: E731
    for bad in (dict(dy=on(z(4, 9))), dict(stats=on(z(2, 4, dtype=F32))), dict(stats=on(z(4, 2))), dict(stats=on(z(4, 4, dtype=F32)[:, :2])),
                dict(add=on(z(4, 8, dtype=F32))), dict(out=on(z(4, 8, dtype=F32)))):
        with pytest.raises(ValueError):
            fp8hg.layernorm_bwd(**ok(**bad))
            pytest.fail(str(bad.keys()))
    for ids in (z(T, dtype=torch.int64), z(2, 3, dtype=torch.int32), z(2 * T, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            fp8hg.lora_plan(on(ids), G)
    for g in (0, 4097):
        with pytest.raises(ValueError):
            fp8hg.lora_plan(on(z(T, dtype=torch.int32)), g)


def test_adapters_that_do_not_fit(gpu0):
    on = gpu0
    call = lambda a=adapters(on), p=plan(on), x=on(z(T, K)), base=on(z(T, N)), **k: fp8hg.lora_add(base, x, a, p, **k)  # noqa: E731
    with pytest.raises(Reached):
        call()
    with pytest.raises(Reached):      # one adapter for all: a stride of 0
        call(fp8hg.LoraAdapters(on(z(1, R, K).expand(G, R, K)), on(z(1, N, R).expand(G, N, R))))
    for bad in (dict(a=fp8hg.LoraAdapters(on(z(G, R, K)), on(z(G, N, R + 1)))), dict(a=fp8hg.LoraAdapters(on(z(G, R, K)), on(z(G + 1, N, R)))),
                dict(a=fp8hg.LoraAdapters(on(z(R, K)), on(z(N, R)))), dict(a=fp8hg.LoraAdapters(on(z(G, R, K, dtype=F32)), on(z(G, N, R)))),
                dict(a=fp8hg.LoraAdapters(on(z(G, K, R).transpose(1, 2)), on(z(G, N, R)))),
                dict(a=adapters(on, scale=lambda t: on(z(G)))), dict(a=adapters(on, ranks=lambda t: on(z(G, dtype=torch.int64)))),
                dict(a=adapters(on, scale=lambda t: on(z(G + 1, dtype=F32)))),
                dict(p=plan(on, T + 1)), dict(p=plan(on, T, G + 1)), dict(x=on(z(T, K + 1))), dict(x=on(z(T, K, dtype=F32))),
                dict(base=on(z(T, N + 1))), dict(base=on(z(T + 1, N))), dict(out=on(z(T, N, dtype=F32))), dict(out_dtype=F32)):
        with pytest.raises(ValueError):
            call(**bad)
            pytest.fail(str(bad.keys()))
    bwd = lambda dy=on(z(T, N)), x=on(z(T, K)), v=on(z(T, R, dtype=F32)), **k: fp8hg.lora_add_bwd(dy, x, v, adapters(on), plan(on), **k)  # noqa: E731
    with pytest.raises(Reached):
        bwd()
    for bad in (dict(dy=on(z(T, N + 1))), dict(dy=on(z(T, N, dtype=F32))), dict(x=on(z(T + 1, K))), dict(v=on(z(T, R))),
                dict(v=on(z(T, R + 1, dtype=F32))), dict(base=on(z(T, N))), dict(params_dtype=torch.float16),
                dict(base=on(z(T, K)), out=on(z(T, K, dtype=F32)))):
        with pytest.raises(ValueError):
            bwd(**bad)
            pytest.fail(str(bad.keys()))


@pytest.mark.parametrize("stride", [0, 1, 99, 4096])
def test_strides_of_one_row_say_nothing(gpu0, stride):
    row = lambda n, dtype=BF16: gpu0(torch.zeros(2 * (n + stride), dtype=dtype).as_strided((1, n), (stride, 1)))  # noqa: E731
    assert adapt._matrix(row(100), "x", adapt._BF16, 0)[1] == 112
    with pytest.raises(Reached):
        fp8hg.layernorm(row(100))
    with pytest.raises(Reached):
        fp8hg.lora_add(row(N), row(K), adapters(gpu0), plan(gpu0, 1))


def test_workspaces_are_asked_for_by_size():
    """The sizes that Python keeps are the library's, of sizes alone."""
    f = adapt._fns()
    adapt._bytes.cache_clear()
    for t, g, r, n, k in ((1, 1, 16, 64, 64), (300, 5, 24, 130, 70), (8192, 1, 64, 8960, 1536), (100, 100, 128, 99, 1)):
        assert adapt._bytes("fp8hg_lora_workspace", t, g, r, k) == f.fp8hg_lora_workspace(t, g, r, k) > 0
        assert adapt._bytes("fp8hg_lora_bwd_workspace", t, g, r, n, k) == f.fp8hg_lora_bwd_workspace(t, g, r, n, k) > 0
        assert adapt._bytes("fp8hg_layernorm_bwd_workspace", t, n) == f.fp8hg_layernorm_bwd_workspace(t, n) > 0
