"""GPU parity of attention over the 8-bit cache behind a prefix that all sequences share, against the definition in 64
bits over each sequence's whole keys (kvq8_ref). Tolerance: that of the attention over the cache (test_gpu_kvq8): the
arithmetic is the same, and a merge of summaries adds a few fp32 roundings, inside its 2^-12."""
import math

import numpy as np
import pytest
import torch

import kvq8_ref as ref
from test_gpu_kvq8 import CODE, DEV, DT, as_ref, filled, ints, random_table, status_ok

pytestmark = pytest.mark.gpu
SPLITS = [(0, 0), (0, 1), (0, 7), (1, 0), (2, 3), (5, 0)]  # (n_splits, n_parts)


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def tables(rng, prefix, lens, page, spare=2):
    """(prefix pages, page table of the sequences, number of pages): the first row is the prefix."""
    t, n = random_table(rng, [prefix, *lens], page, spare)
    shared = t[0, : max(1, (prefix + page - 1) // page)]
    width = max(1, max((n + page - 1) // page for n in lens))
    return shared, t[1:, :width], n


def check(q, cache, shared, prefix, table, lens, out, lse, scale, causal, most=64, rows=slice(None)):
    kc, ks, vc, vs = as_ref(cache)
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    qn, o, l = q.cpu().double().numpy(), out.cpu().double().numpy(), lse.cpu().double().numpy()
    for b, n in enumerate(lens):
        k, v = (np.concatenate([ref.gather(c, s, shared, prefix), ref.gather(c, s, table[b], n)], 1)
                for c, s in ((kc, ks), (vc, vs)))
        want, wl, mag, top, tot = ref.attend(qn[b], k, v, scale, causal)
        assert top.max() <= most
        seen = np.isfinite(wl)
        assert np.array_equal(np.isneginf(l[b]), ~seen)
        assert np.all(o[b][~seen] == 0.0)
        vmax = np.abs(v).max() if v.size else 0.0
        tol = (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -25 * k.shape[1] * vmax / tot[..., None] + half * np.abs(want) + 1e-30
        err = np.abs(o[b] - want)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        if seen.any():
            assert np.all(np.abs(l[b][seen] - wl[seen]) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(wl[seen]))


def call(fa, q, cache, shared, prefix, table, lens, **kw):
    splits = kw.pop("splits", None)
    if splits is not None:
        n = (kw.get("max_prefix") or len(shared) * cache.k_codes.shape[2])
        kw.update(n_splits=min(splits[0], (n + 127) // 128), n_parts=splits[1])
    return fa.attention_kvq8_prefix(q, cache, ints([int(x) for x in shared]), ints([prefix]), ints(table.tolist()), ints(lens), **kw)


CASES = [
    # fmt, dtype, page, H, Hkv, Nq, d, prefix, lens, causal
    ("int8", "bf16", 16, 1, 1, 1, 64, 1, [1], False),
    ("int8", "bf16", 16, 8, 2, 1, 128, 100, [0, 17, 300], False),
    ("e4m3", "fp16", 32, 4, 4, 5, 64, 300, [5, 0, 64, 3], True),
    ("e4m3", "bf16", 64, 16, 1, 1, 128, 0, [257, 0, 511], False),
    ("int8", "fp16", 128, 12, 2, 7, 64, 129, [129, 6, 0], True),
    ("e4m3", "bf16", 16, 40, 1, 16, 128, 17, [15, 16, 70], True),
    ("int8", "bf16", 64, 5, 1, 3, 64, 1999, [2, 1], True),
    ("int8", "fp16", 16, 8, 1, 2, 128, 3, [1, 0, 2], True),
    ("e4m3", "bf16", 128, 8, 8, 1, 128, 1280, [128, 1], False),
    ("e4m3", "fp16", 16, 16, 2, 1, 64, 515, [7] * 40, False),
    ("int8", "bf16", 32, 8, 1, 3, 128, 700, [40, 3, 9] * 5, True),
]


@pytest.mark.parametrize("fmt,dtype,page,H,Hkv,Nq,d,prefix,lens,causal", CASES)
@pytest.mark.parametrize("splits", [None, *SPLITS])
def test_matches_the_definition(fa, fmt, dtype, page, H, Hkv, Nq, d, prefix, lens, causal, splits):
    rng = np.random.default_rng(H * 100 + Nq + prefix + sum(lens))
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    q = torch.from_numpy(rng.standard_normal((len(lens), H, Nq, d))).to(DT[dtype]).to(DEV)
    out, lse = call(fa, q, cache, shared, prefix, table, lens, causal=causal, splits=splits, max_prefix=max(prefix, 1),
                    max_len=max(max(lens), 1))
    status_ok(fa)
    check(q, cache, shared, prefix, table, lens, out, lse, 1 / math.sqrt(d), causal)


@pytest.mark.parametrize("splits", [None, (0, 0), (0, 100), (1, 0), (2, 9), (7, 0)])
@pytest.mark.parametrize("fmt,d", [("int8", 64), ("e4m3", 128)])
def test_many_sequences(fa, fmt, d, splits):
    """More rows than a few tiles, the last one partly filled; with seven runs more CTAs than SMs."""
    rng = np.random.default_rng(d)
    lens = [int(x) for x in rng.integers(0, 70, 301)]
    shared, table, n_pages = tables(rng, 900, lens, 16)
    cache = filled(fa, rng, fmt, n_pages, 2, 16, d)
    q = torch.from_numpy(rng.standard_normal((301, 8, 3, d))).to(torch.bfloat16).to(DEV)
    out, lse = call(fa, q, cache, shared, 900, table, lens, causal=True, splits=splits, max_prefix=900, max_len=max(lens))
    status_ok(fa)
    check(q, cache, shared, 900, table, lens, out, lse, 1 / math.sqrt(d), True)


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("fmt,d", [("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("scale", [0.0, -0.11, 0.4])
def test_scales_and_growing_scores(fa, fmt, d, scale, splits):
    """Scores that grow along the keys move the running maxima; a scale of 0, and a negative one."""
    rng = np.random.default_rng(21)
    page, prefix, lens, H = 32, 2500, [300, 17], 4
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, fmt, n_pages, 2, page, d, exps=(-7, -6))
    order = torch.from_numpy(shared).to(DEV)
    for codes, s in ((cache.k_scale, 1.0), (cache.v_scale, -1.0)):  # K grows, V shrinks along the prefix
        e = torch.linspace(-1, 2, order.numel(), device=DEV).round() * s
        codes[order] = codes[order] * torch.exp2(e)[:, None]
    q = torch.from_numpy(rng.standard_normal((2, H, 3, d))).bfloat16().to(DEV)
    if scale == 0.4:
        q *= 0.5
    out, lse = call(fa, q, cache, shared, prefix, table, lens, scale=scale, causal=True, splits=splits)
    status_ok(fa)
    check(q, cache, shared, prefix, table, lens, out, lse, scale, True)


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("what", ["odd", "zero", "wide"])
def test_page_scales(fa, fmt, dtype, what, splits):
    """Pages of zeros, scales that are no powers of two and up to five orders of magnitude apart (odd), all values or all
    keys of a run zero, and powers of two 2^12 apart that stay exact (wide)."""
    rng = np.random.default_rng(22)
    page, prefix, lens, d = 16, 700, [100, 0, 33], 128
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, fmt, n_pages, 2, page, d)
    if what == "odd":
        cache.v_scale.copy_(torch.from_numpy(10.0 ** rng.uniform(-5, 0, cache.v_scale.shape)).float().to(DEV))
        cache.v_scale[shared[3]] = 0.0
        cache.k_scale[shared[4]] = 0.0
        cache.k_scale[shared[5], 1] = 0.01337
    elif what == "zero":
        cache.v_scale[shared] = 0.0
        cache.k_scale[shared[10:30]] = 0.0
    else:
        for s, top in ((cache.k_scale, -5), (cache.v_scale, 3)):
            e = top - rng.integers(0, 13, s.shape) - (0 if fmt == "int8" else 2)
            s.copy_(torch.from_numpy(2.0 ** e.astype(np.float64)).float().to(DEV))
    q = torch.from_numpy(rng.standard_normal((3, 4, 1, d))).to(DT[dtype]).to(DEV)
    out, lse = call(fa, q, cache, shared, prefix, table, lens, splits=splits)
    status_ok(fa)
    check(q, cache, shared, prefix, table, lens, out, lse, 1 / math.sqrt(d), False)


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("first", ["low", "high"])
def test_small_weights_of_large_values(fa, fmt, first, splits):
    """A page of scores 0 and values near 2^-110, and one of scores -87 (weights near 2^-126) and values near 2^20, which
    make the result: neither a weight nor the quotient of the scales may leave its range on the way. (Bound: the scores are
    single products of up to 126 in log2 units with roundings of 4 2^-24 of itself, inside 2^-12 relative.)"""
    rng = np.random.default_rng(42)
    page, prefix, d = 32, 150, 64
    shared, table, n_pages = tables(rng, prefix, [0], page)
    cache = filled(fa, rng, fmt, n_pages, 1, page, d)
    high = np.array([i % 2 == (first == "low") for i in range(len(shared))])
    k = np.zeros((n_pages, 1, page, d))
    k[shared[high], ..., 0] = -64.0
    cache.k_codes.copy_(torch.from_numpy(k).to(CODE[fmt]).to(DEV))
    cache.k_scale.fill_(87.0 / 64)
    e = np.zeros(n_pages)
    e[shared] = np.where(high, 20.0, -110.0)
    cache.v_scale.copy_(torch.from_numpy(2.0 ** e)[:, None].float().to(DEV))
    q = torch.zeros((1, 2, 3, d), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    out, lse = call(fa, q.to(DEV), cache, shared, prefix, table, [0], scale=1.0, splits=splits)
    status_ok(fa)
    kc, ks, vc, vs = as_ref(cache)
    v = ref.gather(vc, vs, shared, prefix)
    want, wl, mag, _, tot = ref.attend(q[0].double().numpy(), ref.gather(kc, ks, shared, prefix), v, 1.0, False)
    o, l = out[0].cpu().double().numpy(), lse[0].cpu().double().numpy()
    big = np.exp(-87.0) * np.abs(v).max()
    tol = (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -25 * prefix * big / tot[..., None] + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(o - want) <= tol), float((np.abs(o - want) / tol).max())
    assert np.all(np.abs(l - wl) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(wl))


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("fmt,d,Nq", [("int8", 64, 1), ("e4m3", 128, 5)])
def test_rows_of_very_low_scores(fa, fmt, d, Nq, splits):
    """Scores of -1e32 and +1e32, the largest of each row alone, in the prefix or in the sequence's own keys: that value,
    rounded once. (lse: five roundings of one product, below 2^-21 of itself.)"""
    rng = np.random.default_rng(41)
    lens, page, H, prefix = [1, 37, 200, 0], 16, 2, 300
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, fmt, n_pages, 1, page, d)
    k = np.zeros((n_pages, 1, page, d))
    k[..., 0] = 96.0
    k[shared[2], 0, 5, 0] = 64.0   # the key that the rows of low scores are left with
    k[shared[7], 0, 3, 0] = 112.0  # and the one of the high rows
    cache.k_codes.copy_(torch.from_numpy(k).to(CODE[fmt]).to(DEV))
    cache.k_scale.fill_(1.0)
    q = torch.zeros((4, H, Nq, d), dtype=torch.bfloat16)
    q[..., 0] = -1e30
    q[:, 1, Nq // 2 :, 0] = 1e30
    out, lse = call(fa, q.to(DEV), cache, shared, prefix, table, lens, scale=1.0, splits=splits)
    status_ok(fa)
    kc, ks, vc, vs = as_ref(cache)
    o, l = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for b, n in enumerate(lens):
        kk, vv = (np.concatenate([ref.gather(c, s, shared, prefix), ref.gather(c, s, table[b], n)], 1)
                  for c, s in ((kc, ks), (vc, vs)))
        want, wl, *_ = ref.attend(q[b].double().numpy(), kk, vv, 1.0, False)
        assert np.all(np.abs(o[b] - want) <= 2.0 ** -8 * np.abs(want))
        assert np.all(np.abs(l[b] - wl) <= 2.0 ** -21 * np.abs(wl))


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("apart,base", [(10, 0), (22, 0), (32, 0), (32, 95), (32, -118), (0, -110)])
def test_small_elements_beside_an_outlier(fa, apart, base, splits):
    """bf16 rows with one element up to 2^32 times the rest, over keys whose code there is 0: the scores are made of the
    small elements alone, which enter the products exactly."""
    rng = np.random.default_rng(43 + apart + abs(base))
    lens, page, H, d, Nq, prefix = [60, 17], 16, 4, 128, 3, 200
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, "int8", n_pages, 2, page, d)
    x = rng.choice([-1, 1], (2, H, Nq, d)) * (1 + rng.integers(0, 128, (2, H, Nq, d)) / 128)
    dim = rng.integers(0, d, (2, H, Nq))
    np.put_along_axis(x, dim[..., None], 2.0 ** apart, -1)
    x *= 2.0 ** base
    cache.k_codes.view(torch.uint8)[..., torch.from_numpy(np.unique(dim)).to(DEV)] = 0
    q = torch.from_numpy(x).bfloat16()
    scale = 2.0 ** -base / math.sqrt(d)
    out, lse = call(fa, q.to(DEV), cache, shared, prefix, table, lens, scale=scale, splits=splits)
    status_ok(fa)
    check(q, cache, shared, prefix, table, lens, out, lse, scale, False)


@pytest.mark.parametrize("splits", SPLITS)
def test_nan_queries_and_what_lies_behind_the_lengths(fa, splits):
    """A NaN query makes its own row NaN; codes behind the lengths, and pages of nobody, do not matter."""
    rng = np.random.default_rng(7)
    lens, page, prefix = [40, 3, 0], 32, 333
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, "e4m3", n_pages, 2, page, 64)
    q = torch.randn(3, 8, 2, 64, device=DEV).bfloat16()
    q[1, 3, 1, 7], q[2, 6, 0, 0] = float("nan"), float("nan")
    out, lse = call(fa, q, cache, shared, prefix, table, lens, splits=splits)
    nan = torch.isnan(lse)
    assert nan.sum() == 2 and nan[1, 3, 1] and nan[2, 6, 0]
    assert torch.equal(torch.isnan(out), nan[..., None].expand_as(out))
    used = torch.zeros(n_pages, page, dtype=torch.bool, device=DEV)
    for row, n in ((shared, prefix), *((table[b], n) for b, n in enumerate(lens))):
        for t in range(n):
            used[int(row[t // page]), t % page] = True
    for codes in (cache.k_codes, cache.v_codes):
        codes.view(torch.uint8)[(~used)[:, None].expand(n_pages, 2, page)] = 0x7F  # NaN in e4m3
    again, lse2 = call(fa, q, cache, shared, prefix, table, lens, splits=splits)
    assert torch.equal(out[~nan], again[~nan]) and torch.equal(lse[~nan], lse2[~nan])
    status_ok(fa)


@pytest.mark.parametrize("splits", SPLITS)
def test_bad_pages_and_lengths(fa, splits):
    rng = np.random.default_rng(9)
    lens, page, prefix, d = [40, 20], 16, 200, 64
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, "int8", n_pages, 1, page, d)
    q = torch.randn(2, 2, 1, d, device=DEV).half()
    for wrong in (-1, prefix + 1):  # counts as 0
        out, lse = call(fa, q, cache, shared, wrong, table, lens, splits=splits, max_prefix=prefix)
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_ERR_SEQLENS
        check(q, cache, shared, 0, table, lens, out, lse, 0.125, False)
    out, lse = call(fa, q, cache, shared, prefix, table, [40, -3], splits=splits)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_SEQLENS
    check(q, cache, shared, prefix, table, [40, 0], out, lse, 0.125, False)
    # a bad page of the prefix is left out: the same as its neighbours without it
    bad = shared.copy()
    bad[3], bad[12] = n_pages, -1
    out, lse = call(fa, q, cache, bad, prefix, table, lens, splits=splits)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_PAGE
    good = np.delete(shared, [3, 12])
    check(q, cache, good, prefix - 24, table, lens, out, lse, 0.125, False)  # page 12 held 8 tokens


@pytest.mark.parametrize("splits", SPLITS)
def test_guard_bands_streams_graphs_and_repeats(fa, splits):
    rng = np.random.default_rng(11)
    lens, page, prefix, d, H, Nq = [130, 9, 77, 0, 300], 16, 900, 128, 8, 2
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, "int8", n_pages, 2, page, d)
    q = torch.randn(5, H, Nq, d, device=DEV).bfloat16()
    pt, pl, t, n = ints([int(x) for x in shared]), ints([prefix]), ints(table.tolist()), ints(lens)
    n_splits, n_parts = splits
    need = fa.fa_kvq8_prefix_workspace_bytes(5, H, 2, Nq, prefix, d, n_splits, n_parts)
    room = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    rows = 5 * H * Nq
    flat = torch.full((rows * d + 256,), 7.0, dtype=torch.bfloat16, device=DEV)
    fl = torch.full((rows + 128,), 7.0, device=DEV)
    out, lse = flat[128 : 128 + rows * d].view(5, H, Nq, d), fl[64 : 64 + rows].view(5, H, Nq)
    fa.fa_fwd_kvq8_prefix(q, cache, pt, pl, t, n, out, lse, d ** -0.5, True, prefix, 300, n_splits, n_parts, room[256 : 256 + need])
    status_ok(fa)
    assert (room[:256] == 0xA5).all() and (room[256 + need :] == 0xA5).all()
    assert (flat[:128] == 7).all() and (flat[128 + rows * d :] == 7).all() and (fl[:64] == 7).all() and (fl[64 + rows :] == 7).all()
    check(q, cache, shared, prefix, table, lens, out, lse, d ** -0.5, True)
    kw = dict(causal=True, max_prefix=prefix, max_len=300, n_splits=n_splits, n_parts=n_parts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):  # bit for bit
        o2, l2 = fa.attention_kvq8_prefix(q, cache, pt, pl, t, n, stream=side, **kw)
        side.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, l3 = fa.attention_kvq8_prefix(q, cache, pt, pl, t, n, **kw)
    q.copy_(torch.randn_like(q))
    pl.fill_(515)
    n.copy_(ints([100, 0, 77, 250, 1]))
    graph.replay()
    torch.cuda.synchronize()
    check(q, cache, shared, 515, table, [100, 0, 77], o3[:3], l3[:3], d ** -0.5, True)
    assert fa.fa_get_device_status() == fa.FA_ERR_PAGE  # sequence 3 has no pages for its 250 keys
