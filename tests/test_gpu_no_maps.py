"""The adapters without tensor maps: where the driver has no encoder, or refuses a map,
the warps copy what TMA would have, rows that were copied into the plan's order among
it.  The library's own objects, linked with a lookup that finds no encoder."""
import os
import subprocess
import sys

import pytest

from fp8_hybrid_granularity_gb300 import build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
LOOKUP = "_ZN5fp8hg18tensor_map_encoderEv"


def test_adapters_without_tensor_maps(cuda_lib, tmp_path):
    objects = [os.path.join(build.BUILD_DIR, s.replace(".cu", ".o")) for s in build.SOURCES]
    if not all(os.path.exists(o) for o in objects):
        build.build(force=True)
    so = str(tmp_path / "no_maps.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-cudart", "static", "-Xcompiler", "-fPIC", "-Xlinker", f"--wrap={LOOKUP}",
                    "-o", so, os.path.join(HERE, "no_maps.cu"), *objects], check=True)
    # rows of even and odd numbers of columns (the latter copied in the plan's order),
    # tokens of several adapters mixed and some without one
    code = f"""
import sys
sys.path[:0] = [{os.path.dirname(HERE)!r}, {HERE!r}]
from fp8_hybrid_granularity_gb300 import build
build.LIB_PATH, build.is_stale = {so!r}, lambda: False
import torch
import fp8_hybrid_granularity_gb300 as lib
import test_gpu_lora as t
for size in ((300, 256, 520, 24, 5), (300, 1003, 517, 24, 5), (513, 131, 2049, 64, 7), (260, 301, 333, 128, 2)):
    t.test_forward(lib, size, torch.bfloat16)
    t.test_backward(lib, size, torch.bfloat16, torch.float32)
assert lib.fp8hg_get_device_error() == 0
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]
