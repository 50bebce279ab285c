"""GPU tests of the 8-bit key/value cache at the edges of its ranges, against the definitions in 64 bits (kvq8_ref):
scores and page scales of any size, queries of uneven magnitude, scales that no append wrote, and each status by itself."""
import math

import numpy as np
import pytest
import torch

import kvq8_ref as ref
from test_gpu_kvq8 import CODE, DEV, DT, as_ref, check_attention, check_cache, filled, ints, random_table, status_ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


# ---------------------------------------------------------------- scores far below zero
@pytest.mark.parametrize("n_parts", [0, 1, 3])
@pytest.mark.parametrize("fmt,d,Nq", [("int8", 64, 1), ("e4m3", 128, 1), ("int8", 128, 5), ("e4m3", 64, 12)])
def test_attention_rows_of_very_low_scores(fa, fmt, d, Nq, n_parts):
    """Scores of -1e32 and +1e32: a row whose scores are all far below zero still has a largest one, whose value it gets.

    Scores are single products here and every row's largest stands alone, 2^-3 of itself above the next, so the weights are
    1 and 0 and out is one value, rounded once: half a step. lse is one product's roundings, of scale log2 e,
    of the page scale times it, of the score, of ln 2 and the last one: 5 2^-24 of itself, below 2^-21."""
    rng = np.random.default_rng(41)
    lens, page, H = [1, 37, 700, 0], 16, 2
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, fmt, n_pages, 1, page, d)
    k = np.zeros((n_pages, 1, page, d))
    k[..., 0] = 96.0
    for s, n in enumerate(lens):
        if n:
            k[table[s, 0], 0, 0, 0] = 64.0            # the key that the rows of low scores are left with
            if n > 1:
                k[table[s, 1], 0, 3, 0] = 112.0       # and the one of the high rows
    cache.k_codes.copy_(torch.from_numpy(k).to(CODE[fmt]).to(DEV))
    cache.k_scale.fill_(1.0)
    q = torch.zeros((4, H, Nq, d), dtype=torch.bfloat16)
    q[..., 0] = -1e30
    q[:, 1, Nq // 2 :, 0] = 1e30
    out, lse = fa.attention_kvq8(q.to(DEV), cache, ints(table.tolist()), ints(lens), scale=1.0, causal=True,
                                 n_parts=n_parts, max_len=700)
    status_ok(fa)
    kc, ks, vc, vs = as_ref(cache)
    o, l = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for b, n in enumerate(lens):
        want, wl, *_ = ref.attend(q[b].double().numpy(), ref.gather(kc, ks, table[b], n), ref.gather(vc, vs, table[b], n), 1.0, True)
        seen = np.isfinite(wl)
        assert np.array_equal(np.isneginf(l[b]), ~seen) and np.all(o[b][~seen] == 0.0)
        assert np.all(np.abs(o[b] - want) <= 2.0 ** -8 * np.abs(want))
        assert np.all(np.abs(l[b][seen] - wl[seen]) <= 2.0 ** -21 * np.abs(wl[seen]))


# ---------------------------------------------------------------- V scales far apart
@pytest.mark.parametrize("n_parts", [0, 1, 2])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("first", ["low", "high"])
def test_attention_small_weights_of_large_values(fa, fmt, first, n_parts):
    """A page of scores 0 and values near 2^-110, and one of scores -87 (weights near 2^-126) and values near 2^20, which
    make the result: neither a weight nor the quotient of the scales may leave its range on the way.

    Bound: as in check_attention, but the scores are single products of up to 126 in log2 units, each with roundings of
    4 2^-24 of itself: 126 2^-22 ln 2 < 2^-15 relative, inside its 2^-12; no weight is below fp16's normal range against
    the largest contribution but those of the page that is 2^-5 of it, so its second term stays."""
    rng = np.random.default_rng(42)
    page, n, d = 32, 150, 64
    table, n_pages = random_table(rng, [n], page)
    cache = filled(fa, rng, fmt, n_pages, 1, page, d)
    high = np.array([i % 2 == (first == "low") for i in range(table.shape[1])])  # by page: values of 2^20
    k = np.zeros((n_pages, 1, page, d))
    k[table[0][high], ..., 0] = -64.0
    cache.k_codes.copy_(torch.from_numpy(k).to(CODE[fmt]).to(DEV))
    cache.k_scale.fill_(87.0 / 64)
    e = np.zeros(n_pages)
    e[table[0]] = np.where(high, 20.0, -110.0)
    cache.v_scale.copy_(torch.from_numpy(2.0 ** e)[:, None].float().to(DEV))
    q = torch.zeros((1, 2, 3, d), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    out, lse = fa.attention_kvq8(q.to(DEV), cache, ints(table.tolist()), ints([n]), scale=1.0, causal=True, n_parts=n_parts)
    status_ok(fa)
    kc, ks, vc, vs = as_ref(cache)
    v = ref.gather(vc, vs, table[0], n)
    want, wl, mag, _, tot = ref.attend(q[0].double().numpy(), ref.gather(kc, ks, table[0], n), v, 1.0, True)
    o, l = out[0].cpu().double().numpy(), lse[0].cpu().double().numpy()
    big = np.exp(-87.0) * np.abs(v).max()  # the largest contribution's size
    tol = (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -25 * n * big / tot[..., None] + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(o - want) <= tol), float((np.abs(o - want) / tol).max())
    assert np.all(np.abs(l - wl) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(wl))


# ---------------------------------------------------------------- queries of uneven magnitude
@pytest.mark.parametrize("apart,base", [(10, 0), (18, 0), (22, 0), (27, 0), (32, 0), (32, 95), (32, -118), (5, -118), (1, -112),
                                        (0, -110), (20, 60)])
@pytest.mark.parametrize("fmt,d,Nq", [("int8", 64, 1), ("e4m3", 128, 3)])
def test_attention_small_elements_beside_an_outlier(fa, fmt, d, Nq, apart, base):
    """bf16 rows with one element up to 2^32 times the rest, over keys whose code there is 0, anywhere in the type's range:
    the scores are made of the small elements alone, which enter the products exactly (check_attention's bound has no term
    for Q)."""
    rng = np.random.default_rng(43 + apart + abs(base))
    lens, page, H = [200, 17], 16, 4
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, fmt, n_pages, 2, page, d)
    x = rng.choice([-1, 1], (2, H, Nq, d)) * (1 + rng.integers(0, 128, (2, H, Nq, d)) / 128)  # all 8 bits in use, in [1, 2)
    dim = rng.integers(0, d, (2, H, Nq))
    np.put_along_axis(x, dim[..., None], 2.0 ** apart, -1)
    x *= 2.0 ** base
    codes = cache.k_codes.view(torch.uint8)
    codes[..., torch.from_numpy(np.unique(dim)).to(DEV)] = 0
    q = torch.from_numpy(x).bfloat16()
    assert np.array_equal(q.double().numpy(), x)
    for n_parts in (0, 2):
        out, lse = fa.attention_kvq8(q.to(DEV), cache, ints(table.tolist()), ints(lens), n_parts=n_parts,
                                     scale=2.0 ** -base / math.sqrt(d))
        status_ok(fa)
        check_attention(q, cache, table, lens, out, lse, 2.0 ** -base / math.sqrt(d), False)


# ---------------------------------------------------------------- scales that are no powers of two
def halfway(rng, fmt, dtype, scales, shape):
    """16-bit values at or next to the middle between two codes under `scales` (broadcast), of at most half the largest."""
    codes = np.arange(-64.0, 65.0)
    if fmt == "e4m3":
        codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        codes = np.unique(codes[np.abs(codes) <= 224])
    return torch.from_numpy(rng.choice((codes[1:] + codes[:-1]) / 2, shape) * scales).to(DT[dtype])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_to_pages_of_any_scale(fa, fmt, dtype):
    """Pages that hold tokens under scales that are no powers of two: they keep them while these are large enough, and
    codes are x / s rounded once. A scale that is a small odd number times a power of two puts many values exactly in the
    middle, where the even code is due."""
    rng = np.random.default_rng(44)
    page, Hkv, d, n_seq = 16, 2, 64, 100
    held = [int(x) for x in rng.integers(1, page, n_seq)]
    cache = filled(fa, rng, fmt, n_seq, Hkv, page, d)
    s = rng.integers(3, 128, (n_seq, Hkv)) * 2.0 ** -12  # by sequence
    s[::5] = rng.uniform(0.01, 0.02, s[::5].shape).astype(np.float32)
    table = rng.permutation(n_seq)[:, None]
    for scale in (cache.k_scale, cache.v_scale):
        scale[torch.from_numpy(table[:, 0])] = torch.from_numpy(s).float().to(DEV)
    want = as_ref(cache)
    new = [page - h for h in held]
    cu = [0] + [int(c) for c in np.cumsum(new)]
    k, v = (halfway(rng, fmt, dtype, np.repeat(s, new, axis=0)[:, :, None], (cu[-1], Hkv, d)) for _ in range(2))
    fa.kvq8_append(cache, k.to(DEV), v.to(DEV), ints(table.tolist()), ints(cu), ints(held), page)
    for i, x in ((0, k), (2, v)):
        ref.append(want[i], want[i + 1], fmt, x.double().numpy(), table, cu, held)
    assert np.array_equal(want[1][table[:, 0]], s.astype(np.float32))  # none grew
    status_ok(fa)
    check_cache(cache, want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_that_grows_a_scale_of_any_value(fa, fmt):
    """Earlier codes are rounded once to the power of two that a larger new token asks for, whatever their scale was: every
    c s_old / s here is off the middle between two codes by less than fp32 resolves."""
    rng = np.random.default_rng(45)
    page, d, n = 32, 64, 2000
    c0 = np.array([3.0, 5.0, 7.0, 11.0, 13.0, 15.0]) if fmt == "e4m3" else np.arange(3.0, 127.0, 2.0)
    codes = rng.choice(c0, n)
    if fmt == "int8":
        mid = rng.integers(0, codes.astype(int)) + 0.5
    else:
        mid = 2.0 ** rng.integers(-3, 1, n) * (rng.integers(8, 16, n) + 0.5) / 8
    s_old = (mid / codes).astype(np.float32)
    assert np.all((s_old > 0) & (s_old < 1))
    cache = fa.kv_cache_q8(n, 1, page, d, CODE[fmt], DEV)
    for t, s in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        t.copy_(torch.from_numpy(np.broadcast_to(codes[:, None, None, None], t.shape).copy()).to(CODE[fmt]).to(DEV))
        s.copy_(torch.from_numpy(s_old).float()[:, None].to(DEV))
    want = as_ref(cache)
    big = torch.full((n, 1, d), ref.QMAX[fmt], dtype=torch.bfloat16)  # scale 1
    table, cu, held = np.arange(n)[:, None], list(range(n + 1)), [5] * n
    fa.kvq8_append(cache, big.to(DEV), big.to(DEV), ints(table.tolist()), ints(cu), ints(held), 1)
    for i in (0, 2):
        ref.append(want[i], want[i + 1], fmt, big.double().numpy(), table, cu, held)
    status_ok(fa)
    check_cache(cache, want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_read_under_scales_of_any_value(fa, fmt, dtype):
    """code * scale rounded once to the 16-bit type, next to the middle between two of its numbers."""
    rng = np.random.default_rng(46)
    page, d, n = 16, 64, 4000
    bits = 8 if dtype == "bf16" else 11
    c0 = np.array([9.0, 11.0, 13.0, 15.0]) if fmt == "e4m3" else np.arange(3.0, 128.0, 2.0)
    codes = rng.choice(c0, n)
    mid = (rng.integers(2 ** (bits - 1), 2 ** bits, n) + 0.5) * 2.0 ** -bits
    s = (mid / codes).astype(np.float32)
    cache = fa.kv_cache_q8(n, 1, page, d, CODE[fmt], DEV)
    for t, sc in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        t.copy_(torch.from_numpy(np.broadcast_to(codes[:, None, None, None], t.shape).copy()).to(CODE[fmt]).to(DEV))
        sc.copy_(torch.from_numpy(s)[:, None].to(DEV))
    k, v = fa.kvq8_read(cache, ints(np.arange(n)[None].tolist()), ints([0, n * page]), n * page, n * page, dtype=DT[dtype])
    status_ok(fa)
    m, e = np.frexp(codes * s.astype(np.float64))  # the product in 64 bits is exact, and rounded once (torch's conversion
    want = np.ldexp(np.rint(m * 2.0 ** bits), e - bits)  # from 64 bits may go by way of 32)
    want = torch.from_numpy(np.repeat(want, page)).to(DT[dtype])[:, None, None].expand(-1, 1, d)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)


# ---------------------------------------------------------------- each status by itself
BAD_PAGE = [([[0, 1], [2, 99]], [20, 20]), ([[0, 1], [-1, 3]], [20, 20])]
BAD_LEN = [([[0, 1], [2, 3]], [20, 33]), ([[0, 1], [2, 3]], [20, -1])]


@pytest.mark.parametrize("table,held,want", [
    ([[0, 1], [2, 99]], [19, 19], "FA_ERR_PAGE"),
    ([[0, 1], [-1, 3]], [19, 5], "FA_ERR_PAGE"),
    ([[0, 1], [2, 3]], [19, 32], "FA_ERR_SEQLENS"),
    ([[0, 1], [2, 3]], [-1, 19], "FA_ERR_SEQLENS"),
    ([[0, 1], [99, 3]], [19, 19], "FA_OK"),  # an entry that the new token does not need
])
def test_append_reports_what_was_wrong(fa, table, held, want):
    cache = fa.kv_cache_q8(4, 1, 16, 64, torch.int8, DEV)
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16, device=DEV)
    fa.kvq8_append(cache, x, x, ints(table), ints([0, 1, 2]), ints(held), 1)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == getattr(fa, want)
    status_ok(fa)


@pytest.mark.parametrize("table,lens", BAD_PAGE + BAD_LEN[:1])
def test_read_reports_what_was_wrong(fa, table, lens):
    cache = fa.kv_cache_q8(4, 1, 16, 64, torch.int8, DEV)
    cu = [0, lens[0], lens[0] + lens[1]]
    fa.kvq8_read(cache, ints(table), ints(cu), cu[-1], 40)
    torch.cuda.synchronize()
    want = fa.FA_ERR_PAGE if table in [t for t, _ in BAD_PAGE] else fa.FA_ERR_SEQLENS
    assert fa.fa_get_device_status() == want
    # more tokens than max_len, and a first position below 0
    for first, most in ((None, 19), ([0, -1], 20)):
        fa.kvq8_read(cache, ints([[0, 1], [2, 3]]), ints([0, 20, 40]), 40, most, None if first is None else ints(first))
        torch.cuda.synchronize()
        assert fa.fa_get_device_status() == fa.FA_ERR_SEQLENS
    status_ok(fa)


@pytest.mark.parametrize("n_parts", [0, 1, 2, 5])
@pytest.mark.parametrize("table,lens", BAD_PAGE + BAD_LEN)
def test_attention_reports_what_was_wrong(fa, table, lens, n_parts):
    cache = fa.kv_cache_q8(4, 1, 16, 64, torch.int8, DEV)
    q = torch.ones((2, 2, 1, 64), dtype=torch.bfloat16, device=DEV)
    for H in (1, 2):
        fa.attention_kvq8(q[:, :H].contiguous(), cache, ints(table), ints(lens), n_parts=n_parts)
        torch.cuda.synchronize()
        want = fa.FA_ERR_PAGE if table in [t for t, _ in BAD_PAGE] else fa.FA_ERR_SEQLENS
        assert fa.fa_get_device_status() == want
    fa.attention_kvq8(q, cache, ints([[0, 1], [2, 3]]), ints([20, 32]), n_parts=n_parts)
    status_ok(fa)
