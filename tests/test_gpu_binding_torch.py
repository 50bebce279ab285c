"""The binding's allocations on the GPU: with and without torch's private allocator, and under its deterministic mode."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def calls(fa):
    """One call of each kind that allocates, on the current and on another stream."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 2, 64, generator=g).bfloat16().to(DEV)
    cache = fa.kv_cache_q8(6, 2, 16, 64, torch.int8, DEV)
    table, cu, held = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([[0, 1, 2], [3, 4, 5]], [0, 25, 40], [0, 0]))
    fa.kvq8_append(cache, x, x * 2, table, cu, held, 25)
    lens = torch.tensor([25, 15], dtype=torch.int32, device=DEV)
    q = torch.randn(2, 4, 3, 64, generator=g).bfloat16().to(DEV)
    kv = torch.randn(2, 2, 300, 64, generator=g).bfloat16().to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    res = []
    for stream in (None, side, side.cuda_stream):
        res += fa.kvq8_read(cache, table, cu, 40, 25, stream=stream)
        for n_parts in (0, 2):
            res += fa.attention_kvq8(q, cache, table, lens, n_parts=n_parts, stream=stream)
        out, lse = fa.attention_cross(q, kv, kv, n_splits=2, stream=stream)
        res += [out, lse, *fa.attention_cross_backward(q, kv, kv, out, q, lse, stream=stream)[1:]]
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    return res


def test_without_the_private_allocator(fa, monkeypatch):
    want = calls(fa)
    for name in ("_empty_strided_cuda", "_get_device", "_get_raw_stream"):
        if hasattr(fa, name):
            monkeypatch.setattr(fa, name, None)
    got = calls(fa)
    assert all(a.shape == b.shape and a.dtype == b.dtype and a.device == b.device and torch.equal(a, b)
               for a, b in zip(want, got))


def test_rows_that_nothing_writes_are_filled_under_deterministic_algorithms(fa):
    """torch fills what torch.empty gives with NaN while deterministic algorithms are on; so do the binding's outputs."""
    cache = fa.kv_cache_q8(1, 1, 16, 64, torch.int8, DEV)
    table, cu = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([[0]], [0, 5]))
    junk = torch.full((200, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    del junk
    torch.use_deterministic_algorithms(True)
    try:
        k, v = fa.kvq8_read(cache, table, cu, 200, 5)
    finally:
        torch.use_deterministic_algorithms(False)
    assert bool((k[:5] == 0).all()) and bool((v[:5] == 0).all())
    assert bool(torch.isnan(k[5:]).all()) and bool(torch.isnan(v[5:]).all())
