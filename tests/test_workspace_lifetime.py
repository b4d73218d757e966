"""A call's workspace lives until the library has returned: the interpreter's lock
is free during a call, and memory that nobody refers to is another thread's next
tensor.  Without a GPU: the library and its tensors are stood in for."""
import weakref

import pytest
import torch

import fp8_hybrid_granularity_gb300 as fp8hg
from fp8_hybrid_granularity_gb300 import adapt, lowbit
from test_lowbit_refusals import StandIn

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def alive(monkeypatch):
    """Whether the last workspace was there during the library's call: a list of answers."""
    answers, last = [], []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_workspace") or name.endswith("_bytes"):
                    return 4096
                answers.append(last[-1]() is not None)
                return 0
            return call

    def scratch(n, x, stream):
        t = StandIn(torch.empty(n, dtype=torch.uint8))
        last.append(weakref.ref(t))
        return t

    monkeypatch.setattr(lowbit, "_cuda_device", lambda: 0)
    monkeypatch.setattr(lowbit, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(lowbit, "_fns", Library)
    monkeypatch.setattr(lowbit, "_new", lambda *a: StandIn(torch.empty_strided(*a[:2], dtype=a[2])), raising=False)
    monkeypatch.setattr(lowbit, "_scratch", scratch)
    monkeypatch.setattr(adapt, "_fns", Library)
    monkeypatch.setattr(adapt, "_bound", None)
    monkeypatch.setattr(adapt, "_new", lambda *a: StandIn(torch.empty_strided(*a[:2], dtype=a[2])))
    adapt._bytes.cache_clear()
    yield answers
    adapt._bytes.cache_clear()


def z(*shape, dtype=BF16):
    return StandIn(torch.zeros(shape, dtype=dtype))


T, N, K, R, G = 6, 24, 16, 8, 2


def adapters():
    return fp8hg.LoraAdapters(z(G, R, K), z(G, N, R))


def plan():
    return fp8hg.LoraPlan(z(64, dtype=torch.int32), T, G)


CALLS = {
    "layernorm_bwd": lambda: fp8hg.layernorm_bwd(z(4, 8), z(4, 8), None, z(4, 2, dtype=F32)),
    "lora_add": lambda: fp8hg.lora_add(None, z(T, K), adapters(), plan()),
    "lora_add_bwd": lambda: fp8hg.lora_add_bwd(z(T, N), z(T, K), z(T, R, dtype=F32), adapters(), plan()),
    "fp4_tensor_scale": lambda: fp8hg.fp4_tensor_scale(z(4, 64)),
    "fp4_linear": lambda: fp8hg.fp4_linear(z(40, 64), fp8hg.Fp4Tensor(z(32, 32, dtype=torch.uint8), z(1024, dtype=torch.uint8), 32, 64, fp8hg.FP4_MX)),
}


@pytest.mark.parametrize("name", CALLS)
def test_workspace_outlives_the_call(alive, name):
    CALLS[name]()
    assert alive == [True]
