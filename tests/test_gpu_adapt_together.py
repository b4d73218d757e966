"""The layer norm's and adapters' calls beside one another: threads on one stream and on
streams of their own, graphs that share a pool, a first call under capture."""
import pathlib
import subprocess
import sys
import threading

import pytest
import torch

from test_gpu_lora import adapters, batch, rand

pytestmark = pytest.mark.gpu


def step(lib, s, w, b, base):
    """Norm, adapters, and back: workspaces below and above what a thread keeps."""
    y, stats = lib.layernorm(s["x"], w, b)
    plan = lib.lora_plan(s["ids"], s["a"].shape[0])
    z, v = lib.lora_add(base, y, adapters(lib, s), plan, keep=True)
    dx, da, db = lib.lora_add_bwd(s["dy"], y, v, adapters(lib, s), plan)
    return (z, v, da, db) + lib.layernorm_bwd(dx, s["x"], w, stats, add=dx)


def inputs(size, seed):
    s = batch(*size, seed=seed)
    k = size[2]
    return s, 1 + 0.1 * rand(seed + 90, k), 0.1 * rand(seed + 91, k), rand(seed + 92, size[0], size[1]).bfloat16()


SIZES = [(1500, 1003, 520, 24, 5), (40, 264, 136, 16, 12), (700, 512, 2048, 64, 3), (1, 264, 520, 8, 2)]


@pytest.mark.parametrize("own_streams", [False, True])
def test_threads(cuda_lib, own_streams):
    """Every thread's results are those of its calls alone, on one stream (where memory
    given back by one thread is the other's next) and on streams of their own."""
    jobs = [inputs(size, 300 + 10 * i) for i, size in enumerate(SIZES)]
    want = [step(cuda_lib, *j) for j in jobs]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def run(i):
        try:
            stream = torch.cuda.Stream() if own_streams else torch.cuda.default_stream()
            with torch.cuda.stream(stream):
                for _ in range(40):
                    got = step(cuda_lib, *jobs[i])
                    if not all(torch.equal(p, q) for p, q in zip(got, want[i])):
                        wrong.append(i)
        except Exception as e:      # noqa: BLE001 - reported by the test
            errors.append(repr(e))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and not wrong
    assert cuda_lib.fp8hg_get_device_error() == 0


def test_graphs_of_one_pool(cuda_lib):
    """Two graphs whose memory is one pool's, replayed in turn with new inputs."""
    jobs = [inputs(size, 400 + 10 * i) for i, size in enumerate(SIZES[:2])]
    new = [inputs(size, 500 + 10 * i) for i, size in enumerate(SIZES[:2])]
    want = [step(cuda_lib, *j) for j in new]
    for j in jobs:
        step(cuda_lib, *j)
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], torch.cuda.graph_pool_handle()
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(step(cuda_lib, *j))
        graphs.append(g)
    for (s, *rest), (s2, *rest2) in zip(jobs, new):
        for name in s:
            s[name].copy_(s2[name])
        for p, q in zip(rest, rest2):
            p.copy_(q)
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(got, w))


@pytest.mark.parametrize("call", ["norm", "fp8", "adapters", "few"])
def test_first_call_of_a_process_captured(cuda_lib, call):
    """What a kernel's first call looks up and asks for is allowed under capture."""
    code = f"""
import torch
import fp8_hybrid_granularity_gb300 as lib
x, dy = torch.randn(300, 1000, device="cuda").bfloat16(), torch.randn(300, 512, device="cuda").bfloat16()
ids = torch.randint(-1, 3, (300,), device="cuda").int()
w = lib.LoraAdapters(torch.randn(3, 16, 1000, device="cuda").bfloat16(), torch.randn(3, 512, 16, device="cuda").bfloat16())
def norm():
    y, stats = lib.layernorm(x)
    return (y, stats) + lib.layernorm_bwd(x, x, None, stats)
def fp8():
    q, y, stats = lib.fp8_layernorm(x, group=128, with_y=True)
    return q.codes, q.scales(), y, stats
def adapters():
    plan = lib.lora_plan(ids, 3)
    y, v = lib.lora_add(None, x, w, plan, keep=True)
    return (y, v) + lib.lora_add_bwd(dy, x, v, w, plan)
def few():
    return lib.lora_add(None, x[:4], w, lib.lora_plan(ids[:4], 3), keep=True)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = {call}()
graph.replay()
want = {call}()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(out, want))
"""
    root = pathlib.Path(__file__).resolve().parent.parent
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
