"""The time limit of the waits between a kernel's own warps, on a barrier that
nobody completes (the kernels' arrivals are unconditional: in them it never runs out)."""
import ctypes
import os
import subprocess

import pytest
import torch

from fp8_hybrid_granularity_gb300 import build

pytestmark = pytest.mark.gpu


def test_wait_ends_at_its_limit(cuda_lib, tmp_path):
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "wait_limit.cu")
    so = str(tmp_path / "wait_limit.so")
    subprocess.run([build._nvcc(), "-std=c++17", *build.ARCH, "-O3", "-shared", "-Xcompiler", "-fPIC", src, "-o", so],
                   check=True)
    run = ctypes.CDLL(so).wait_limit
    run.argtypes = [ctypes.c_uint, ctypes.c_void_p]
    for limit in (1_000_000, 30_000_000):
        out = torch.zeros(3, dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        assert run(limit, out.data_ptr()) == 0
        gave_up, longest, done = out.tolist()
        # a try may suspend the warp for a while past the limit
        assert gave_up == 4 and limit <= longest < limit + 100_000_000 and done == 4
