"""Adapters at the edges of what a call may be given: non-finite values beside
ranks."""
import pytest
import torch

import adapt_ref as ref
from test_gpu_lora import adapters, batch, rand

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
