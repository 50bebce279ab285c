"""GPU parity of the forward over keys of another length, and of its gradients, for one to three query rows and several
heads to a group, as in generation over an encoder's states; against 64 bits, within test_gpu_cross's bounds."""
import math

import numpy as np
import pytest
import torch

from test_gpu_cross import check, inputs, ints, reference, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


@pytest.mark.parametrize("dtype,B,H,Hkv,Nq,Nk,d", [
    ("bf16", 5, 16, 2, 1, 700, 128),   # groups of 8
    ("fp16", 4, 10, 2, 1, 333, 64),    # 5
    ("bf16", 3, 12, 3, 1, 1500, 64),   # 4
    ("fp16", 3, 8, 1, 3, 257, 128),    # 8
    ("bf16", 20, 8, 2, 1, 130, 128),   # more units than half the SMs
    ("fp16", 40, 8, 2, 2, 129, 64),    # more units than SMs
])
def test_few_rows_of_grouped_heads(fa, dtype, B, H, Hkv, Nq, Nk, d):
    rng = np.random.default_rng(Nk)
    lens = [Nk, 0, 1][:B] + [int(x) for x in rng.integers(0, Nk + 1, max(0, B - 3))]
    q, k, v, do = inputs(Nk, dtype, B, H, Hkv, Nq, Nk, d)
    ref = reference(q, k, v, lens, 1 / math.sqrt(d), do)
    for n_splits in (None, 1, min(3, (Nk + 127) // 128)):
        out, lse = fa.attention_cross(q, k, v, ints(lens), n_splits=n_splits)
        status_ok(fa)
        check("out", out, ref["out"])
        check("lse", lse, ref["lse"])
    got = fa.attention_cross_backward(q, k, v, out, do, lse, ints(lens))
    status_ok(fa)
    for name, t in zip(("dq", "dk", "dv"), got):
        check(name, t, ref[name])
