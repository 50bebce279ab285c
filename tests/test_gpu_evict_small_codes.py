"""GPU: eviction of tokens whose codes are small beside a larger one that set their page's scale and goes. The new scale is
then far below the old one (2^17 times for e4m3's smallest code), and the codes are multiplied by as much, rounded once.
What is left is compared for equality with the definition."""
import numpy as np
import pytest
import torch

import evict_ref as er
from test_gpu_kvq8 import CODE, DEV, as_ref, check_cache, ints, random_table, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


SMALL = {"int8": [1.0, 2.0, 5.0], "e4m3": [2.0 ** -9, 3 * 2.0 ** -9, 2.0 ** -6, 0.09375, 0.4375, 0.875]}


@pytest.mark.parametrize("scales", ["powers", "odd", "apart"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("page,d", [(16, 64), (32, 128), (128, 64), (64, 128)])
def test_small_codes_beside_an_evicted_outlier(fa, fmt, page, d, scales):
    """Every fourth position is the outlier, and has the least weight. The others hold codes up to a bound of their
    page, one of e4m3's smallest or int8's 1 among them; some hold zeros."""
    rng = np.random.default_rng(page + d)
    lens, Hkv = [11 * page + 5, 3, 7 * page], 2
    table, n_pages = random_table(rng, lens, page)
    cache = fa.kv_cache_q8(n_pages, Hkv, page, d, CODE[fmt], DEV)
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        most = rng.choice(SMALL[fmt], (n_pages, Hkv, 1, 1))
        unit = 1.0 if fmt == "int8" else 2.0 ** -9
        x = np.minimum(np.floor(rng.random(codes.shape) * (most / unit + 1)), most / unit) * unit
        x = np.where(rng.random(codes.shape[:3])[..., None] < 0.05, 0.0, x) * rng.choice([-1.0, 1.0], codes.shape)
        x = torch.from_numpy(x).to(CODE[fmt]).double().numpy()  # (0.4375 + 2^-9 steps: to a code, below the bound or at it)
        x[:, :, ::4] = rng.choice([-1.0, 1.0], x[:, :, ::4].shape) * (127.0 if fmt == "int8" else 448.0)
        codes.copy_(torch.from_numpy(x).to(CODE[fmt]).to(DEV))
        e = rng.integers(-60, 60, scale.shape) if scales == "apart" else np.full(scale.shape, -3)
        s = 2.0 ** e.astype(np.float64) * (1.37 if scales == "odd" else 1.0)
        scale.copy_(torch.from_numpy(s).float().to(DEV))
    cap = table.shape[1] * page
    w = rng.random((len(lens), Hkv, cap)).astype(np.float32) + 1
    w[:, :, ::4] = 0.0
    keep = 5 * page + 3
    at = [[er.keep_positions(w[s, h, :n], keep, 0) for h in range(Hkv)] for s, n in enumerate(lens)]
    want = as_ref(cache)
    for i in (0, 2):
        er.evict(want[i], want[i + 1], fmt, table, lens, at)
    _, kept, _ = fa.kvq8_evict(cache, ints(table.tolist()), ints(lens), torch.from_numpy(w).to(DEV), keep, 0)
    status_ok(fa)
    assert kept[0, 0].tolist() == at[0][0]
    check_cache(cache, want)


@pytest.mark.parametrize("odd", [1.0, 1.37])
@pytest.mark.parametrize("code", [2.0 ** -9, 2.0 ** -8, 7 * 2.0 ** -9, 2.0 ** -4, 0.4375, 0.5, 0.875, 1.0])
def test_one_code_alone(fa, code, odd):
    """All values of the tokens kept are one code: they keep their value, to e4m3's rounding under the new scale."""
    page, d, n = 16, 64, 48
    cache = fa.kv_cache_q8(3, 1, page, d, CODE["e4m3"], DEV)
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        x = torch.full(codes.shape, code, dtype=torch.float64)
        x[:, :, 1] = 448.0
        codes.copy_(x.to(CODE["e4m3"]).to(DEV))
        scale.fill_(odd)
    value = code * float(cache.k_scale[0, 0])
    w = torch.ones(1, 1, n, device=DEV)
    w[..., 1::16] = 0.0
    fa.kvq8_evict(cache, ints([[2, 0, 1]]), ints([n]), w, 45, 0)
    status_ok(fa)
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        x = codes.cpu().float().double() * scale.cpu().double()[..., None, None]
        for p, held in ((2, 16), (0, 16), (1, 13)):
            assert (x[p, 0, :held] - value).abs().max() <= 2.0 ** -4 * value
            assert float(scale[p, 0]) <= value / 224
