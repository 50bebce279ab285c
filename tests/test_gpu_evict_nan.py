"""GPU: eviction by weights of which more are NaN than there are places, beside weights above 0 only. NaN counts as the
greatest, of equal ones the lower position is kept, and nothing is written around the outputs."""
import numpy as np
import pytest
import torch

import evict_ref as er
from test_gpu_kvq8 import DEV, as_ref, check_cache, filled, ints, random_table, status_ok

pytestmark = pytest.mark.gpu
GUARD = 4096


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def guarded(shape, dtype, value):
    """A tensor with GUARD elements of `value` on either side, and those."""
    n = int(np.prod(shape))
    flat = torch.full((n + 2 * GUARD,), value, dtype=dtype, device=DEV)
    return flat[GUARD : GUARD + n].view(shape), (flat[:GUARD], flat[GUARD + n :])


CASES = [
    # lens, keep, recent, what is NaN of the earlier positions
    ([1050, 30], 1000, 100, "first"),
    ([2000], 300, 299, "some"),
    ([1000, 1000], 100, 0, "half"),
    ([700, 1, 900], 17, 3, "all"),
    ([400] * 5, 399, 1, "half"),
    ([27000], 5000, 40, "half"),
    ([27000], 20000, 1, "some"),
]


@pytest.mark.parametrize("lens,keep,recent,what", CASES)
@pytest.mark.parametrize("fmt,page,Hkv,d", [("int8", 16, 3, 64), ("e4m3", 128, 2, 128)])
def test_more_nan_than_places(fa, lens, keep, recent, what, fmt, page, Hkv, d):
    rng = np.random.default_rng(sum(lens) + keep)
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    cap = table.shape[1] * page
    w = np.exp(rng.standard_normal((len(lens), Hkv, cap))).astype(np.float32)
    for s, n in enumerate(lens):
        old = max(n - recent, 0)
        if what == "first":
            w[s, :, : max(old - 50, 0)] = np.nan
        elif what == "all":
            w[s, :, :old] = np.nan
        else:
            w[s, :, :old][rng.random((Hkv, old)) < (0.5 if what == "half" else 0.07)] = np.nan
    at = [[er.keep_positions(w[s, h, :n], keep, recent) for h in range(Hkv)] for s, n in enumerate(lens)]
    want = as_ref(cache)
    for i in (0, 2):
        er.evict(want[i], want[i + 1], fmt, table, lens, at)
    lens_out, g0 = guarded((len(lens),), torch.int32, 77)
    kept, g1 = guarded((len(lens), Hkv, keep), torch.int32, 77)
    out, g2 = guarded(w.shape, torch.float32, 7.0)
    fa.kvq8_evict(cache, ints(table.tolist()), ints(lens), torch.from_numpy(w).to(DEV), keep, recent, lens_out, kept, out)
    status_ok(fa)
    for g, value in ((g0, 77), (g1, 77), (g2, 7)):
        assert all((x == value).all() for x in g)
    assert lens_out.tolist() == [min(n, keep) for n in lens]
    for s in range(len(lens)):
        for h in range(Hkv):
            m = len(at[s][h])
            assert kept[s, h].tolist() == at[s][h] + [-1] * (keep - m)
            assert np.array_equal(out[s, h, :m].cpu().numpy(), w[s, h][at[s][h]], equal_nan=True)
            assert (out[s, h, m:] == 0).all()
    check_cache(cache, want)
