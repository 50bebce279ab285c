"""GPU parity of the 8-bit cache's weights and eviction against the definitions in 64 bits (evict_ref).

What an eviction leaves is compared for equality: the choice orders numbers, scales are powers of two, and a code is one
rounding. The weights' tolerance is derived in evict_ref.weights."""
import numpy as np
import pytest
import torch

import evict_ref as er
import kvq8_ref as ref
from test_gpu_kvq8 import CODE, DEV, DT, as_ref, check_cache, filled, ints, numbers, random_table, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


# ---------------------------------------------------------------- weights
WEIGHTS = [
    # fmt, dtype, page, H, Hkv, Nq, d, lens, causal
    ("int8", "bf16", 16, 2, 2, 1, 64, [1], False),
    ("int8", "bf16", 16, 8, 2, 1, 128, [0, 17, 300], False),
    ("e4m3", "fp16", 32, 4, 4, 5, 64, [3, 5, 64, 999], True),
    ("e4m3", "bf16", 64, 16, 1, 1, 128, [257, 0, 511], False),
    ("int8", "fp16", 128, 12, 2, 7, 64, [129, 6], True),
    ("e4m3", "bf16", 16, 40, 1, 16, 128, [15, 16, 700], True),
    ("int8", "bf16", 64, 5, 1, 3, 64, [2, 1, 1300], False),
    ("e4m3", "fp16", 16, 4, 2, 2, 64, [3, 0, 40, 17, 1] * 30, True),
    # rows that share a head: around each number of tiles of eight, and of passes
    *[("int8", ("bf16", "fp16")[rows % 2], 16, 2 * rows, 2, 1, d, [37, 200], False)
      for rows in (8, 9, 16, 17, 24, 25, 32, 33, 48, 49, 64, 72, 80, 129) for d in (64, 128)],
]


@pytest.mark.parametrize("fmt,dtype,page,H,Hkv,Nq,d,lens,causal", WEIGHTS)
def test_weights_match_the_definition(fa, fmt, dtype, page, H, Hkv, Nq, d, lens, causal):
    rng = np.random.default_rng(sum(lens) + H)
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    q = torch.from_numpy(rng.standard_normal((len(lens), H, Nq, d))).to(DT[dtype]).to(DEV)
    t, n = ints(table.tolist()), ints(lens)
    cap = table.shape[1] * page
    _, lse = fa.attention_kvq8(q, cache, t, n, causal=causal)
    weight = torch.from_numpy(rng.random((len(lens), Hkv, cap)) * 3).float().to(DEV)
    before = weight.cpu().double().numpy()
    fa.kvq8_weights(q, cache, t, n, lse, weight, causal=causal, max_len=max(lens))
    status_ok(fa)
    got = weight.cpu().double().numpy()
    kc, ks, _, _ = as_ref(cache)
    for s, m in enumerate(lens):
        assert np.array_equal(got[s, :, m:], before[s, :, m:])  # positions not held
        if m == 0:
            continue
        k = ref.gather(kc, ks, table[s], m)
        add, bound = er.weights(q[s].cpu().double().numpy(), k, lse[s].cpu().double().numpy(), d ** -0.5, causal)
        want = before[s, :, :m] + add
        assert np.all(np.abs(got[s, :, :m] - want) <= bound + 2.0 ** -24 * want)
        if not causal or m >= Nq:  # each row gives away a weight of 1
            assert np.allclose((got[s, :, :m] - before[s, :, :m]).sum(-1), H // Hkv * Nq, rtol=1e-3)


def test_weights_of_rows_without_keys_and_nan(fa):
    """Causal rows of a sequence shorter than they are see nothing and add nothing; a NaN query makes its head's weights
    NaN and no other's."""
    rng = np.random.default_rng(0)
    table, n_pages = random_table(rng, [4, 40], 16)
    cache = filled(fa, rng, "int8", n_pages, 2, 16, 64)
    q = torch.randn(2, 4, 6, 64, device=DEV).bfloat16()
    q[1, 3, 2, 7] = float("nan")
    t, n = ints(table.tolist()), ints([4, 40])
    _, lse = fa.attention_kvq8(q, cache, t, n, causal=True)
    assert torch.isneginf(lse[0, :, :2]).all() and torch.isnan(lse[1, 3, 2])
    weight = torch.zeros(2, 2, table.shape[1] * 16, device=DEV)
    fa.kvq8_weights(q, cache, t, n, lse, weight, causal=True)
    status_ok(fa)
    assert torch.allclose(weight[0].sum(-1), torch.full((2,), 8.0, device=DEV), rtol=1e-3)
    assert torch.isfinite(weight[1, 0]).all() and torch.isnan(weight[1, 1, :37]).all()


def test_weights_bad_lengths_and_pages(fa):
    rng = np.random.default_rng(1)
    table, n_pages = random_table(rng, [40, 40, 40], 16)
    cache = filled(fa, rng, "e4m3", n_pages, 1, 16, 64)
    q = torch.randn(3, 2, 1, 64, device=DEV).half()
    lse = torch.full((3, 2, 1), 3.0, device=DEV)
    for lens, code in (([40, -1, 40], fa.FA_ERR_SEQLENS), ([40, 49, 40], fa.FA_ERR_SEQLENS)):
        w = torch.zeros(3, 1, 48, device=DEV)
        fa.kvq8_weights(q, cache, ints(table.tolist()), ints(lens), lse, w)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == code
        assert (w[1] == 0).all() and (w[0, 0, :40] > 0).all() and (w[2, 0, :40] > 0).all()
    bad = table.copy()
    bad[1, 1] = n_pages
    w = torch.zeros(3, 1, 48, device=DEV)
    fa.kvq8_weights(q, cache, ints(bad.tolist()), ints([40] * 3), lse, w)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_PAGE
    assert (w[1, 0, 16:32] == 0).all() and (w[1, 0, :16] > 0).all() and (w[1, 0, 32:40] > 0).all()


# ---------------------------------------------------------------- eviction
EVICT = [
    # fmt, page, Hkv, d, lens, keep, recent
    ("int8", 16, 1, 64, [2], 1, 0),
    ("int8", 16, 2, 64, [0, 1, 16, 17, 50], 16, 4),
    ("e4m3", 32, 3, 128, [100, 33, 32, 64], 33, 33),
    ("e4m3", 64, 2, 64, [700, 5, 200], 130, 0),
    ("int8", 128, 2, 128, [128, 129, 900], 128, 1),
    ("int8", 16, 5, 128, [1000, 1500], 999, 100),
    ("e4m3", 16, 1, 128, [513, 2000, 77], 300, 299),
    ("int8", 32, 2, 64, [400], 500, 10),
    ("e4m3", 128, 1, 64, [1111, 640], 515, 17),
]


def make_weights(rng, nseq, Hkv, cap, kind):
    w = np.exp(rng.standard_normal((nseq, Hkv, cap)) * 2).astype(np.float32)
    if kind == "ties":
        w = rng.integers(0, 4, w.shape).astype(np.float32) - 1.0
    elif kind == "same":
        w[:] = 0.25
    elif kind == "odd":
        w.reshape(-1)[rng.integers(0, w.size, w.size // 5)] = -0.0
        w.reshape(-1)[rng.integers(0, w.size, w.size // 7)] = 0.0
        for x in (np.nan, np.inf, -np.inf, -3.5, 1e-42, np.float32(3e38)):
            w.reshape(-1)[rng.integers(0, w.size, w.size // 11)] = x
    return w


def run_evict(fa, cache, fmt, table, lens, w, keep, recent):
    want = as_ref(cache)
    before = w.copy()
    weight = torch.from_numpy(w).to(DEV)
    new, kept, out = fa.kvq8_evict(cache, ints(table.tolist()), ints(lens), weight, keep, recent)
    at = [[er.keep_positions(before[s, h, :n], keep, recent) for h in range(w.shape[1])] for s, n in enumerate(lens)]
    assert np.array_equal(weight.cpu().numpy(), before, equal_nan=True)
    assert new.tolist() == [min(n, keep) for n in lens]
    for s in range(len(lens)):
        for h in range(w.shape[1]):
            m = len(at[s][h])
            assert kept[s, h].tolist() == at[s][h] + [-1] * (keep - m)
            assert np.array_equal(out[s, h, :m].cpu().numpy(), before[s, h][at[s][h]], equal_nan=True)
            assert (out[s, h, m:] == 0).all()
    er.evict(want[0], want[1], fmt, table, lens, at)
    er.evict(want[2], want[3], fmt, table, lens, at)
    return want


@pytest.mark.parametrize("fmt,page,Hkv,d,lens,keep,recent", EVICT)
@pytest.mark.parametrize("kind", ["spread", "ties", "same", "odd"])
def test_evict_matches_the_definition(fa, fmt, page, Hkv, d, lens, keep, recent, kind):
    rng = np.random.default_rng(sum(lens) + keep)
    table, n_pages = random_table(rng, [max(n, 1) for n in lens], page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d, exps=(-9, -3))
    w = make_weights(rng, len(lens), Hkv, table.shape[1] * page, kind)
    want = run_evict(fa, cache, fmt, table, lens, w, keep, recent)
    status_ok(fa)
    check_cache(cache, want)  # every slot of every page: untouched ones as they were


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_evict_scales_far_apart(fa, fmt):
    """Pages under scales 2^200 apart, of zeros, and that are no powers of two; zeros under a scale far above their page's."""
    rng = np.random.default_rng(5)
    page, lens = 16, [400, 333]
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, fmt, n_pages, 2, page, 64, exps=(-100, 100))
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        scale[rng.integers(0, n_pages, 6)] = 0.0
        scale[rng.integers(0, n_pages, 8)] *= 1.37
        codes.view(torch.uint8)[rng.integers(0, n_pages, 8)] = 0
        codes.view(torch.uint8)[:, :, 3] = 0
    w = make_weights(rng, 2, 2, table.shape[1] * page, "spread")
    want = run_evict(fa, cache, fmt, table, lens, w, 171, 20)
    status_ok(fa)
    check_cache(cache, want)


@pytest.mark.parametrize("n,keep,recent", [(8200, 4000, 100), (10000, 9999, 3), (12000, 5000, 500), (12288, 1, 0), (16384, 9000, 5), (16390, 16385, 0), (40000, 100, 99), (40000, 33333, 1), (24577, 24500, 7)])
@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_evict_long_sequences(fa, n, keep, recent, kind):
    rng = np.random.default_rng(n + keep)
    table, n_pages = random_table(rng, [n, 50], 16)
    cache = filled(fa, rng, "int8", n_pages, 1, 16, 64)
    w = make_weights(rng, 2, 1, table.shape[1] * 16, kind)
    want = run_evict(fa, cache, "int8", table, [n, 50], w, keep, recent)
    status_ok(fa)
    check_cache(cache, want)


def test_evict_many_heads(fa):
    """More units than the GPU holds at once."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(1, 300, 90)]
    table, n_pages = random_table(rng, lens, 32)
    cache = filled(fa, rng, "e4m3", n_pages, 8, 32, 64)
    w = make_weights(rng, 90, 8, table.shape[1] * 32, "spread")
    want = run_evict(fa, cache, "e4m3", table, lens, w, 120, 30)
    status_ok(fa)
    check_cache(cache, want)


@pytest.mark.parametrize("count", [128, 129, 300])
@pytest.mark.parametrize("page", [16, 128])
def test_evict_many_sequences(fa, count, page):
    """Up to 128 sequences those that are cut come first, more go by their own place; none, some and long ones cut."""
    rng = np.random.default_rng(count + page)
    lens = [int(x) for x in rng.integers(0, 90, count)]
    lens[:3] = [600, 40, 41]
    table, n_pages = random_table(rng, [max(n, 1) for n in lens], page)
    cache = filled(fa, rng, "int8", n_pages, 2, page, 64)
    w = make_weights(rng, count, 2, table.shape[1] * page, "spread")
    want = run_evict(fa, cache, "int8", table, lens, w, 40, 9)
    status_ok(fa)
    check_cache(cache, want)


def test_evict_bad_lengths_and_pages(fa):
    rng = np.random.default_rng(2)
    lens, page = [100, 100, 100], 16
    table, n_pages = random_table(rng, lens, page)
    w = make_weights(rng, 3, 2, table.shape[1] * page, "spread")
    for wrong in (-5, table.shape[1] * page + 1):
        cache = filled(fa, rng, "int8", n_pages, 2, page, 64)
        given = [100, wrong, 100]
        want = as_ref(cache)
        new, kept, out = fa.kvq8_evict(cache, ints(table.tolist()), ints(given), torch.from_numpy(w).to(DEV), 50, 10)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_ERR_SEQLENS
        assert new.tolist() == [50, 0, 50] and (kept[1] == -1).all() and (out[1] == 0).all()
        at = [[er.keep_positions(w[s, h, :n], 50, 10) for h in range(2)] for s, n in enumerate([100, 0, 100])]
        er.evict(want[0], want[1], "int8", table, [100, 0, 100], at)
        er.evict(want[2], want[3], "int8", table, [100, 0, 100], at)
        check_cache(cache, want)
    # a bad page: tokens from it become zeros, tokens for it are lost, the other sequences are as they should be
    cache = filled(fa, rng, "int8", n_pages, 2, page, 64)
    want = as_ref(cache)
    bad = table.copy()
    bad[1, 2], bad[1, 5] = -1, n_pages + 7
    fa.kvq8_evict(cache, ints(bad.tolist()), ints(lens), torch.from_numpy(w).to(DEV), 50, 10)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_PAGE
    at = [[er.keep_positions(w[s, h, :100], 50, 10) for h in range(2)] for s in range(3)]
    for codes, scales in ((0, 1), (2, 3)):
        held = want[codes][table[1, 2]].copy(), want[scales][table[1, 2]].copy()
        want[codes][table[1, 2]], want[codes][table[1, 5]] = 0.0, 0.0
        other = want[codes].copy(), want[scales].copy()
        er.evict(want[codes], want[scales], "int8", table, lens, at)
        want[codes][table[1, 2]], want[scales][table[1, 2]] = held
    got = as_ref(cache)
    skip = {int(table[1, 5])}
    rows = [p for p in range(n_pages) if p not in skip]
    for i in range(4):
        assert np.array_equal(got[i][rows], want[i][rows])


def test_evict_streams_graphs_and_repeats(fa):
    rng = np.random.default_rng(3)
    lens, page = [300, 210, 90], 32
    table, n_pages = random_table(rng, lens, page)
    first = filled(fa, rng, "int8", n_pages, 2, page, 128)
    w = torch.from_numpy(make_weights(rng, 3, 2, table.shape[1] * page, "spread")).to(DEV)
    t, n = ints(table.tolist()), ints(lens)

    def copy():
        return fa.KVCacheQ8(*(x.clone() for x in first))

    a, b, c = copy(), copy(), copy()
    want = fa.kvq8_evict(a, t, n, w, 100, 30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.kvq8_evict(b, t, n, w, 100, 30, stream=side)
    side.synchronize()
    for x, y in zip((*want, *a), (*got, *b)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.kvq8_evict(c, t, n, w, 100, 30)
    for _ in range(2):
        for x, y in zip(c, first):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((*want, *a), (*got, *c)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    status_ok(fa)


def test_evict_then_append_and_attend(fa):
    """A decoding loop under a budget: what is attended to after an eviction is the kept tokens, and appending goes on."""
    rng = np.random.default_rng(6)
    H, Hkv, d, page, budget = 4, 2, 64, 16, 60
    nseq, cap = 3, 96
    table, n_pages = random_table(rng, [cap] * nseq, page)
    t = ints(table.tolist())
    cache = fa.kv_cache_q8(n_pages, Hkv, page, d, CODE["int8"], DEV)
    weight = torch.zeros(nseq, Hkv, cap, device=DEV)
    lens = torch.zeros(nseq, dtype=torch.int32, device=DEV)
    cu = ints(list(range(nseq + 1)))
    held = [[[] for _ in range(Hkv)] for _ in range(nseq)]  # token numbers, as the cache should hold them
    for step in range(100):
        x = torch.randn(2, nseq, Hkv, d, device=DEV).bfloat16()
        fa.kvq8_append(cache, x[0], x[1], t, cu, lens, 1)
        lens = lens + 1
        q = torch.randn(nseq, H, 1, d, device=DEV).bfloat16()
        out, lse = fa.attention_kvq8(q, cache, t, lens)
        fa.kvq8_weights(q, cache, t, lens, lse, weight)
        for s in range(nseq):
            for h in range(Hkv):
                held[s][h].append(step)
        if int(lens[0]) > budget + 20:
            before = weight.cpu().numpy()
            lens, kept, weight = fa.kvq8_evict(cache, t, lens, weight, budget, 10)
            for s in range(nseq):
                for h in range(Hkv):
                    at = er.keep_positions(before[s, h, : budget + 21], budget, 10)
                    assert kept[s, h].tolist() == at
                    held[s][h] = [held[s][h][i] for i in at]
    assert lens.tolist() == [len(held[0][0])] * nseq and len(held[0][0]) <= budget + 20
    total = weight.sum(-1)
    assert (total > 0).all()
    status_ok(fa)
