"""GPU parity of the 8-bit key/value cache: appending tokens, reading them back, and attention over the cache,
against the definitions in 64 bits (kvq8_ref).

Codes and scales are compared for equality: the scales are powers of two, so a code is one rounding of an exact
quotient. Reading is one rounding of an exact product, so equality again.

Tolerance of the attention, per output element, from the arithmetic. The softmax weights are rounded to fp16:
2^-11 relative, or 2^-25 of the largest weight where they fall below fp16's normal range; the exponentials, the
scores (fp32 sums of at most 128 products, |score| up to S) and the fp32 accumulation are within 2^-13 relative
for the S <= 64 used here (d/2 * 2^-24 * S + 2^-21 is 2.5e-4 at the most pessimistic); the output is rounded
once, half a step of its type. So
    |o - ref| <= (2^-11 + 2^-12) sum_j p_j |v_j| + 2^-25 n max|v| / sum_j exp(s_j - max) + half_step |ref| + 1e-30
and |lse - ref| <= 2^-13 + 2^-22 |lse|.
"""
import math

import numpy as np
import pytest
import torch

import kvq8_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def numbers(codes):
    """Codes as the numbers they stand for, in 64 bits on the CPU."""
    return codes.cpu().float().double().numpy()


def raw(codes):
    return codes.view(torch.uint8).cpu().numpy()


def random_table(rng, caps, page, spare=2):
    """Page table of sequences with room for caps[s] tokens, pages in random order; unused entries are out of range."""
    need = [(c + page - 1) // page for c in caps]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(caps), max(max(need), 1)), 2**30, dtype=np.int64)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at : at + n]
        at += n
    return table, sum(need) + spare


def filled(fa, rng, fmt, n_pages, Hkv, page, d, exps=(-6, -4), mag=1.0):
    """A cache of random codes (every byte of it valid) under random power-of-two scales."""
    c = fa.kv_cache_q8(n_pages, Hkv, page, d, CODE[fmt], DEV)
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        x = rng.standard_normal(codes.shape) * (27.0 if fmt == "int8" else 90.0) * mag
        codes.copy_(torch.from_numpy(ref.round_code(x, fmt)).to(CODE[fmt]).to(DEV))
        e = rng.integers(exps[0], exps[1] + 1, scale.shape) - (0 if fmt == "int8" else 2)
        scale.copy_(torch.from_numpy(2.0 ** e.astype(np.float64)).float().to(DEV))
    return c


def as_ref(cache):
    return [numbers(cache.k_codes), cache.k_scale.cpu().double().numpy(), numbers(cache.v_codes),
            cache.v_scale.cpu().double().numpy()]


def check_cache(cache, want):
    assert np.array_equal(cache.k_scale.cpu().double().numpy(), want[1])
    assert np.array_equal(cache.v_scale.cpu().double().numpy(), want[3])
    assert np.array_equal(numbers(cache.k_codes), want[0])
    assert np.array_equal(numbers(cache.v_codes), want[2])


def status_ok(fa):
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


# ---------------------------------------------------------------- append
APPEND = [
    # fmt, dtype, page, Hkv, d, held, new
    ("int8", "bf16", 16, 2, 128, [0], [1]),
    ("int8", "fp16", 16, 1, 64, [5, 16, 15, 0], [1, 1, 1, 1]),
    ("e4m3", "bf16", 32, 3, 64, [31, 0, 7], [2, 0, 33]),
    ("e4m3", "fp16", 64, 2, 128, [0, 63, 64], [129, 1, 64]),
    ("int8", "bf16", 128, 1, 128, [127, 200], [300, 3]),
    ("int8", "fp16", 64, 5, 64, [1], [62]),
    ("e4m3", "bf16", 16, 2, 128, [3, 0], [500, 17]),
    ("e4m3", "bf16", 128, 2, 64, [0, 0], [0, 130]),
]


@pytest.mark.parametrize("fmt,dtype,page,Hkv,d,held,new", APPEND)
@pytest.mark.parametrize("mul", [1.0, 30.0])
def test_append_matches_the_definition(fa, fmt, dtype, page, Hkv, d, held, new, mul):
    rng = np.random.default_rng(page + Hkv + sum(new))
    table, n_pages = random_table(rng, [a + b for a, b in zip(held, new)], page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    want = as_ref(cache)
    t = sum(new)
    # K and V inside a wider buffer: strides between tokens and heads are not those of a packed tensor
    qkv = torch.from_numpy(rng.standard_normal((t, 2 * Hkv + 1, d + 8)) * mul).to(DT[dtype]).to(DEV)
    k, v = qkv[:, 1 : 1 + Hkv, 8:], qkv[:, 1 + Hkv :, :d]
    cu = [0] + [int(c) for c in np.cumsum(new)]
    fa.kvq8_append(cache, k, v, ints(table.tolist()), ints(cu), ints(held), max(new))
    ref.append(want[0], want[1], fmt, k.cpu().double().numpy(), table, cu, held)
    ref.append(want[2], want[3], fmt, v.cpu().double().numpy(), table, cu, held)
    status_ok(fa)
    check_cache(cache, want)  # every slot of every page: untouched ones as they were


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_extreme_values(fa, fmt, dtype):
    """Zeros, the type's largest and smallest numbers, exact borders of the scales, token by token."""
    big = float(torch.finfo(DT[dtype]).max)
    q = ref.QMAX[fmt]
    tiny = 2.0 ** -133 if dtype == "bf16" else 2.0 ** -24
    rows = [0.0, 0.0, tiny, -0.0, q * 2.0 ** -9, q * 2.0 ** -9 * 1.01, 1.0, -q, q * 1.01, 3.0, big, -big, 0.5, 0.0, 7.0,
            2.0 ** -10, 0.0, tiny, 5.5, q]
    rng = np.random.default_rng(1)
    table, n_pages = random_table(rng, [len(rows)], 16)
    cache = fa.kv_cache_q8(n_pages, 1, 16, 64, CODE[fmt], DEV)
    want = as_ref(cache)
    for i, r in enumerate(rows):
        x = torch.from_numpy(rng.uniform(-1, 1, (1, 1, 64)) * abs(r)).to(DT[dtype])
        x[0, 0, i] = r
        y = x.flip(-1).contiguous()
        fa.kvq8_append(cache, x.to(DEV), y.to(DEV), ints(table.tolist()), ints([0, 1]), ints([i]), 1)
        ref.append(want[0], want[1], fmt, x.double().numpy(), table, [0, 1], [i])
        ref.append(want[2], want[3], fmt, y.double().numpy(), table, [0, 1], [i])
        check_cache(cache, want)
    status_ok(fa)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_token_by_token_stays_within_a_step(fa, fmt):
    """A page filled one token at a time rounds its codes again when its scale grows: by less than one step of the
    final scale in all (half a step for the code, then halves of it for each doubling)."""
    rng = np.random.default_rng(7)
    page, d = 64, 128
    x = torch.from_numpy(rng.standard_normal((page, 1, d)) * np.exp2(np.arange(page) / 6.0)[:, None, None]).bfloat16()
    cache = fa.kv_cache_q8(1, 1, page, d, CODE[fmt], DEV)
    for i in range(page):
        t = x[i : i + 1].to(DEV)
        fa.kvq8_append(cache, t, t, ints([[0]]), ints([0, 1]), ints([i]), 1)
    status_ok(fa)
    s = float(cache.k_scale[0, 0])
    got = numbers(cache.k_codes)[0, 0] * s
    want = x[:, 0].double().numpy()
    if fmt == "int8":
        assert np.abs(got - want).max() <= s
    else:  # half a step of the value (2^-4 of it), or one step of the smallest numbers (2^-9)
        assert np.all(np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, s * 2.0 ** -9))


def test_append_reports_values_no_code_stands_for(fa):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((20, 2, 64))).half()
    x[3, 0, 5], x[4, 1, 6], x[18, 0, 63] = float("inf"), float("nan"), float("-inf")
    cache = fa.kv_cache_q8(2, 2, 16, 64, torch.int8, DEV)
    want = as_ref(cache)
    fa.kvq8_append(cache, x.to(DEV), x.to(DEV), ints([[1, 0]]), ints([0, 20]), ints([0]), 20)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_VALUE
    for i in (0, 2):
        ref.append(want[i], want[i + 1], "int8", x.double().numpy(), [[1, 0]], [0, 20], [0])
    check_cache(cache, want)


def test_append_bad_tables_and_lengths_leave_the_rest_alone(fa):
    """A sequence with a bad length is not written, a bad page's tokens are left out, the others are as usual."""
    rng = np.random.default_rng(4)
    page, Hkv, d, fmt = 16, 2, 64, "e4m3"
    new, held = [20, 20, 20, 20, 20], [0, -1, 4, 30, 8]
    table = np.array([[0, 1, 2], [3, 4, 5], [6, 99, 7], [8, 9, 10], [11, -5, 12]])
    cache = filled(fa, rng, fmt, 13, Hkv, page, d)
    want = as_ref(cache)
    x = torch.from_numpy(rng.standard_normal((100, Hkv, d))).bfloat16()
    cu = [0, 20, 40, 60, 80, 100]
    args = (ints(table.tolist()), ints(cu), ints(held), 20)
    fa.kvq8_append(cache, x.to(DEV), x.to(DEV), *args)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() in (fa.FA_ERR_SEQLENS, fa.FA_ERR_PAGE)
    xs = x.double().numpy()
    for i in (0, 2):
        ref.append(want[i], want[i + 1], fmt, xs[:20], table[:1], [0, 20], [0])
        ref.append(want[i], want[i + 1], fmt, xs[40:52], table[2:3], [0, 12], [4])  # up to the bad page
        ref.append(want[i], want[i + 1], fmt, xs[80:88], table[4:5], [0, 8], [8])
    # held[3] + 20 = 50 tokens do not fit three pages
    check_cache(cache, want)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("fmt,dtype,page,Hkv,d,first,n", [
    ("int8", "bf16", 16, 2, 128, None, [1]),
    ("int8", "fp16", 32, 1, 64, [3, 40, 0], [70, 0, 5]),
    ("e4m3", "bf16", 64, 3, 64, None, [64, 63, 65, 200]),
    ("e4m3", "fp16", 128, 2, 128, [127, 1], [130, 300]),
    ("e4m3", "bf16", 16, 5, 128, [0], [333]),
])
def test_read_gives_the_values_back(fa, fmt, dtype, page, Hkv, d, first, n):
    rng = np.random.default_rng(page + d + sum(n))
    start = first or [0] * len(n)
    table, n_pages = random_table(rng, [a + b for a, b in zip(start, n)], page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    total = sum(n) + 3  # rows behind the last sequence
    cu = [0] + [int(c) for c in np.cumsum(n)]
    k = torch.full((total, Hkv, d), 7.0, dtype=DT[dtype], device=DEV)
    v = k.clone()
    fa.kvq8_read(cache, ints(table.tolist()), ints(cu), total, max(n), None if first is None else ints(first),
                 DT[dtype], k, v)
    status_ok(fa)
    for got, codes, scale in ((k, cache.k_codes, cache.k_scale), (v, cache.v_codes, cache.v_scale)):
        want = np.concatenate([ref.gather(numbers(codes), scale.cpu().double().numpy(), table[s], a + c)[:, a:]
                               .transpose(1, 0, 2) for s, (a, c) in enumerate(zip(start, n))])
        want = torch.from_numpy(want).to(DT[dtype])
        assert torch.equal(got[: sum(n)].cpu(), want)
        assert bool((got[sum(n) :] == 7.0).all())


def test_read_leaves_out_bad_pages_and_lengths(fa):
    rng = np.random.default_rng(5)
    cache = filled(fa, rng, "int8", 4, 1, 16, 64)
    k = torch.full((60, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    v = k.clone()
    fa.kvq8_read(cache, ints([[0, 4], [1, 2], [3, 3]]), ints([0, 20, 25, 60]), 60, 40, None, torch.bfloat16, k, v)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() in (fa.FA_ERR_PAGE, fa.FA_ERR_SEQLENS)
    want = torch.from_numpy(ref.gather(numbers(cache.k_codes), cache.k_scale.cpu().double().numpy(), [0], 16)[0])
    assert torch.equal(k[:16, 0].cpu(), want.bfloat16())
    assert bool((k[16:20] == 9.0).all()) and bool((k[25:] == 9.0).all())  # page 4; 35 tokens in two pages
    want = torch.from_numpy(ref.gather(numbers(cache.k_codes), cache.k_scale.cpu().double().numpy(), [1], 5)[0])
    assert torch.equal(k[20:25, 0].cpu(), want.bfloat16())


# ---------------------------------------------------------------- attention
def check_attention(q, cache, table, lens, out, lse, scale, causal):
    kc, ks, vc, vs = as_ref(cache)
    half = 2.0 ** -8 if q.dtype == torch.bfloat16 else 2.0 ** -11
    qn, o, l = q.cpu().double().numpy(), out.cpu().double().numpy(), lse.cpu().double().numpy()
    for b, n in enumerate(lens):
        k, v = ref.gather(kc, ks, table[b], n), ref.gather(vc, vs, table[b], n)
        want, wl, mag, top, tot = ref.attend(qn[b], k, v, scale, causal)
        assert top.max() <= 64
        seen = np.isfinite(wl)
        assert np.array_equal(np.isneginf(l[b]), ~seen)
        assert np.all(o[b][~seen] == 0.0)
        vmax = np.abs(v).max() if v.size else 0.0
        tol = (2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -25 * n * vmax / tot[..., None] + half * np.abs(want) + 1e-30
        err = np.abs(o[b] - want)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        if seen.any():
            assert np.all(np.abs(l[b][seen] - wl[seen]) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(wl[seen]))


ATTEND = [
    # fmt, dtype, page, H, Hkv, Nq, d, lens, causal, n_parts
    ("int8", "bf16", 16, 1, 1, 1, 64, [1], False, None),
    ("int8", "bf16", 16, 8, 2, 1, 128, [509, 16, 17, 0], False, None),
    ("e4m3", "fp16", 64, 4, 4, 1, 64, [64, 63, 65], False, 1),
    ("e4m3", "bf16", 32, 8, 1, 1, 128, [1000, 31], False, 7),
    ("int8", "fp16", 128, 6, 3, 5, 64, [700, 3, 5, 0, 128], True, None),
    ("e4m3", "bf16", 16, 16, 2, 1, 64, [2000], True, None),
    ("e4m3", "fp16", 64, 10, 2, 3, 128, [777, 2, 1], True, 13),
    ("int8", "bf16", 64, 4, 1, 16, 128, [16, 15, 300, 1], True, 4),
    ("int8", "fp16", 16, 40, 1, 1, 128, [333], False, None),
    ("e4m3", "bf16", 32, 9, 3, 7, 64, [4100, 64], False, None),
    ("int8", "bf16", 16, 2, 2, 2, 128, [9000], True, 3),   # more than 32 tiles for a warp
    ("e4m3", "fp16", 128, 2, 1, 1, 64, [8200, 130], False, 2),
]


@pytest.mark.parametrize("fmt,dtype,page,H,Hkv,Nq,d,lens,causal,n_parts", ATTEND)
def test_attention_matches_the_definition(fa, fmt, dtype, page, H, Hkv, Nq, d, lens, causal, n_parts):
    rng = np.random.default_rng(H * 100 + Nq + sum(lens))
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    q = torch.from_numpy(rng.standard_normal((len(lens), H, Nq, d))).to(DT[dtype]).to(DEV)
    out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints(lens), causal=causal, n_parts=n_parts,
                                 max_len=max(lens))
    status_ok(fa)
    check_attention(q, cache, table, lens, out, lse, 1 / math.sqrt(d), causal)


@pytest.mark.parametrize("fmt,d", [("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("scale", [0.0, -0.11, 0.4])
def test_attention_scales_and_growing_scores(fa, fmt, d, scale):
    """Scores that grow along the keys move the running maxima of both the sum and the weights."""
    rng = np.random.default_rng(21)
    page, n, H = 32, 3000, 4
    table, n_pages = random_table(rng, [n], page)
    cache = filled(fa, rng, fmt, n_pages, 2, page, d, exps=(-7, -6))
    order = torch.from_numpy(table[0]).to(DEV)
    for codes, s in ((cache.k_scale, 1.0), (cache.v_scale, -1.0)):  # K grows, V shrinks along the sequence
        e = torch.linspace(-1, 2, order.numel(), device=DEV).round() * s
        codes[order] = codes[order] * torch.exp2(e)[:, None]
    q = torch.from_numpy(rng.standard_normal((1, H, 3, d))).bfloat16().to(DEV)
    if scale == 0.4:
        q *= 0.5
    out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints([n]), scale=scale, causal=True, n_parts=3)
    status_ok(fa)
    check_attention(q, cache, table, [n], out, lse, scale, True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attention_page_scales_far_apart(fa, fmt, dtype):
    """Pages of zeros (scale 0), and scales that are no powers of two, five orders of magnitude apart."""
    rng = np.random.default_rng(22)
    page, n, d = 16, 400, 128
    table, n_pages = random_table(rng, [n], page)
    cache = filled(fa, rng, fmt, n_pages, 2, page, d)
    cache.v_scale.copy_(torch.from_numpy(10.0 ** rng.uniform(-5, 0, cache.v_scale.shape)).float().to(DEV))
    cache.v_scale[table[0, 3]] = 0.0
    cache.k_scale[table[0, 4]] = 0.0
    cache.k_scale[table[0, 5], 1] = 0.01337
    q = torch.from_numpy(rng.standard_normal((1, 4, 1, d))).to(DT[dtype]).to(DEV)
    for n_parts in (0, 1, 4):
        out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints([n]), n_parts=n_parts)
        status_ok(fa)
        check_attention(q, cache, table, [n], out, lse, 1 / math.sqrt(d), False)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_attention_pages_of_zeros_before_keys_a_row_does_not_see(fa, fmt):
    """Early causal rows that see nothing but values of zero, then tiles in which they see no key."""
    rng = np.random.default_rng(31)
    table, n_pages = random_table(rng, [60], 16)
    cache = filled(fa, rng, fmt, n_pages, 1, 16, 64)
    cache.v_scale[table[0, :3]] = 0.0
    q = torch.from_numpy(rng.standard_normal((1, 2, 16, 64))).half().to(DEV)
    for n_parts in (0, 1, 2):
        out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints([60]), causal=True, n_parts=n_parts)
        status_ok(fa)
        check_attention(q, cache, table, [60], out, lse, 0.125, True)


def test_attention_all_values_zero_and_wide_queries(fa):
    rng = np.random.default_rng(23)
    table, n_pages = random_table(rng, [100], 16)
    cache = filled(fa, rng, "e4m3", n_pages, 1, 16, 64)
    cache.v_scale.zero_()
    q = torch.from_numpy(rng.standard_normal((1, 3, 1, 64))).bfloat16().to(DEV)
    out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints([100]))
    check_attention(q, cache, table, [100], out, lse, 0.125, False)
    assert bool((out == 0).all())
    # query magnitudes far outside fp16's range, brought back by the scale
    big = filled(fa, rng, "int8", n_pages, 1, 16, 64)
    q = torch.from_numpy(rng.standard_normal((1, 3, 1, 64)) * np.array([1e30, 1e25, 1.0])[:, None, None] * 1e-2).bfloat16()
    q = q.to(DEV)
    out, lse = fa.attention_kvq8(q, big, ints(table.tolist()), ints([100]), scale=2.0 ** -100)
    check_attention(q, big, table, [100], out, lse, 2.0 ** -100, False)
    status_ok(fa)


def test_attention_ignores_what_lies_behind_the_lengths(fa):
    """NaN codes in slots past a sequence's end, NaN scales in pages no sequence owns, table entries no token needs."""
    rng = np.random.default_rng(24)
    lens, page, d = [37, 100, 0, 5], 16, 128
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, "e4m3", n_pages, 2, page, d)
    clean = fa.KVCacheQ8(*[t.clone() for t in cache])
    for codes in (cache.k_codes, cache.v_codes):
        bytes_ = codes.view(torch.uint8)
        for s, n in enumerate(lens):
            if n % page:
                bytes_[table[s, n // page], :, n % page :] = 0x7F
    used = set(int(p) for row, n in zip(table, lens) for p in row[: (n + page - 1) // page])
    for p in range(n_pages):
        if p not in used:
            cache.k_scale[p] = cache.v_scale[p] = float("nan")
    for Nq, causal in ((1, False), (6, True)):
        q = torch.from_numpy(rng.standard_normal((4, 4, Nq, d))).half().to(DEV)
        out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints(lens), causal=causal)
        status_ok(fa)
        check_attention(q, clean, table, lens, out, lse, 1 / math.sqrt(d), causal)


@pytest.mark.parametrize("n_parts", [0, 1, 2])
def test_attention_bad_pages_and_lengths(fa, n_parts):
    """Keys of a page that is none are left out; a length out of range counts as 0."""
    rng = np.random.default_rng(25)
    page, d = 16, 64
    cache = filled(fa, rng, "int8", 12, 1, page, d)
    table = np.array([[0, 1, 2, 3], [4, 5, 77, 6], [7, 8, 9, 10], [-1, 11, 11, 11]])
    q = torch.from_numpy(rng.standard_normal((4, 2, 1, d))).bfloat16().to(DEV)
    out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints([64, 60, 65, 10]), n_parts=n_parts)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() in (fa.FA_ERR_PAGE, fa.FA_ERR_SEQLENS)
    check_attention(q[:1], cache, table[:1], [64], out[:1], lse[:1], 1 / 8, False)
    check_attention(q[1:2], cache, [[4, 5, 6]], [44], out[1:2], lse[1:2], 1 / 8, False)  # 32 keys and 12 of page 6
    for b in (2, 3):
        assert bool((out[b] == 0).all()) and bool(torch.isneginf(lse[b]).all())
    status_ok(fa)


def test_attention_repeats_bit_for_bit_and_part_counts_agree(fa):
    rng = np.random.default_rng(26)
    lens, page, d = [3000, 700], 64, 128
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, "int8", n_pages, 2, page, d)
    q = torch.from_numpy(rng.standard_normal((2, 8, 1, d))).bfloat16().to(DEV)
    for n_parts in (0, 1, 2, 5, 47, 3000):
        got = [fa.attention_kvq8(q, cache, ints(table.tolist()), ints(lens), n_parts=n_parts, max_len=3000)
               for _ in range(2)]
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        check_attention(q, cache, table, lens, *got[0], 1 / math.sqrt(d), False)
    status_ok(fa)


@pytest.mark.parametrize("n_parts", [0, 1, 3, 40, 500])
def test_attention_many_sequences_of_uneven_lengths(fa, n_parts):
    """Runs of empty sequences, more sequences than a warp looks at in one go, parts that end anywhere."""
    rng = np.random.default_rng(32)
    page, d, H, Hkv = 16, 64, 6, 2
    lens = [int(x) for x in rng.integers(0, 60, 150)]
    lens[:5] = [0, 0, 33, 0, 1]
    lens[60:100] = [0] * 40
    lens[-3:] = [0, 200, 0]
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, "int8", n_pages, Hkv, page, d)
    q = torch.from_numpy(rng.standard_normal((len(lens), H, 2, d))).half().to(DEV)
    out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints(lens), causal=True, n_parts=n_parts, max_len=200)
    status_ok(fa)
    check_attention(q, cache, table, lens, out, lse, 1 / 8, True)


@pytest.mark.parametrize("fmt,dtype,page,H,Hkv,Nq,d,n_seq,longest,causal", [
    ("int8", "bf16", 16, 8, 8, 1, 64, 6, 1500, False),     # eight CTAs for a unit, warps without tiles
    ("e4m3", "fp16", 64, 12, 2, 7, 128, 7, 2100, True),    # several row tiles
    ("int8", "fp16", 32, 40, 5, 4, 64, 5, 700, True),
    ("e4m3", "bf16", 128, 32, 8, 1, 128, 15, 400, False),  # four
    ("int8", "bf16", 16, 16, 8, 2, 64, 26, 300, True),     # two
    ("e4m3", "fp16", 16, 8, 8, 1, 64, 60, 120, True),      # one
])
def test_attention_with_several_ctas_for_a_unit(fa, fmt, dtype, page, H, Hkv, Nq, d, n_seq, longest, causal):
    """One launch, the CTAs of a unit merging through each other's shared memory: lengths of nothing, one token, one tile,
    as many tiles as warps, one more, and any; the same bits every time."""
    rng = np.random.default_rng(H * n_seq + d)
    lens = [longest, 0, 1, 16, 17][:n_seq] + [int(x) for x in rng.integers(0, longest + 1, max(0, n_seq - 5))]
    lens[-1] = min(longest, 512 if n_seq % 2 else 513)
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    q = torch.from_numpy(rng.standard_normal((n_seq, H, Nq, d))).to(DT[dtype]).to(DEV)
    got = [fa.attention_kvq8(q, cache, ints(table.tolist()), ints(lens), causal=causal, n_parts=0, max_len=longest)
           for _ in range(2)]
    status_ok(fa)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    check_attention(q, cache, table, lens, *got[0], 1 / math.sqrt(d), causal)
    q[0, H - 1, Nq - 1, 3] = float("nan")  # a NaN query gives NaN, and only its own row
    out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints(lens), causal=causal, n_parts=0, max_len=longest)
    status_ok(fa)
    assert bool(out[0, H - 1, Nq - 1].isnan().all()) and bool(lse[0, H - 1, Nq - 1].isnan())
    keep = torch.ones(n_seq, H, Nq, dtype=torch.bool, device=DEV)
    keep[0, H - 1, Nq - 1] = False
    assert torch.equal(out[keep], got[0][0][keep]) and torch.equal(lse[keep], got[0][1][keep])


def test_attention_nothing_cached(fa):
    cache = fa.kv_cache_q8(4, 2, 32, 128, torch.float8_e4m3fn, DEV)
    q = torch.ones((3, 4, 1, 128), dtype=torch.bfloat16, device=DEV)
    table = ints([[0, 1], [2, 3], [0, 0]])
    for n_parts in (0, 1, 7):
        out, lse = fa.attention_kvq8(q, cache, table, ints([0, 0, 0]), n_parts=n_parts)
        status_ok(fa)
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_attention_guard_bands(fa):
    """Nothing is written outside out, lse and the workspace; a row that is NaN stays its own."""
    rng = np.random.default_rng(33)
    lens, page, d = [900, 31], 32, 128
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, "e4m3", n_pages, 1, page, d)
    q = torch.from_numpy(rng.standard_normal((2, 3, 5, d))).bfloat16().to(DEV)
    q[0, 1, 2, 3] = float("nan")
    n = q.numel()
    for n_parts in (0, 1, 9):
        nb = fa.fa_kvq8_workspace_bytes(3, 1, 5, d, n_parts)
        bo = torch.full((n + 8192,), 3.0, dtype=q.dtype, device=DEV)
        bl = torch.full((30 + 2048,), 3.0, device=DEV)
        ws = torch.full((nb + 1024,), 7, dtype=torch.uint8, device=DEV)
        out, lse = bo[4096 : 4096 + n].view(q.shape), bl[1024 : 1024 + 30].view(2, 3, 5)
        fa.fa_fwd_kvq8(q, cache, ints(table.tolist()), ints(lens), out, lse, 0.1, False, 900, n_parts, ws[:nb])
        status_ok(fa)
        assert bool((bo[:4096] == 3.0).all()) and bool((bo[4096 + n :] == 3.0).all())
        assert bool((bl[:1024] == 3.0).all()) and bool((bl[1024 + 30 :] == 3.0).all())
        assert bool((ws[nb:] == 7).all())
        assert bool(torch.isnan(out[0, 1, 2]).all()) and bool(torch.isnan(lse[0, 1, 2]))
        clean = q.clone()
        clean[0, 1, 2] = 0
        out[0, 1, 2] = 0
        kept = torch.ones((2, 3, 5), dtype=torch.bool, device=DEV)
        kept[0, 1, 2] = False
        want, wl = fa.attention_kvq8(clean, cache, ints(table.tolist()), ints(lens), scale=0.1, max_len=900, n_parts=n_parts)
        assert torch.equal(out[kept], want[kept]) and torch.equal(lse[kept], wl[kept])
        check_attention(clean, cache, table, lens, want, wl, 0.1, False)


def test_attention_offsets_past_32_bits(fa):
    """Pages more than 2^32 bytes into the cache."""
    page, Hkv, d = 128, 4, 128
    n_pages = (1 << 32) // (page * Hkv * d) + 70
    cache = fa.KVCacheQ8(*[torch.empty((n_pages, Hkv, page, d), dtype=torch.int8, device=DEV) for _ in range(2)],
                         *[torch.zeros((n_pages, Hkv), device=DEV) for _ in range(2)])
    rng = np.random.default_rng(27)
    table = (n_pages - 1 - rng.permutation(60)[:4])[None]
    x = torch.from_numpy(rng.standard_normal((400, Hkv, d))).bfloat16().to(DEV)
    fa.kvq8_append(cache, x, x * 0.5, ints(table.tolist()), ints([0, 400]), ints([0]), 400)
    k, v = fa.kvq8_read(cache, ints(table.tolist()), ints([0, 400]), 400, 400)
    assert float((k.float() - x.float()).abs().max()) <= 0.5 * float(cache.k_scale.max())
    assert float((v.float() - x.float() * 0.5).abs().max()) <= 0.5 * float(cache.v_scale.max())
    q = torch.from_numpy(rng.standard_normal((1, 4, 1, d))).bfloat16().to(DEV)
    out, lse = fa.attention_kvq8(q, cache, ints(table.tolist()), ints([400]))
    status_ok(fa)
    top = table.min()
    small = fa.KVCacheQ8(*[t[top:].contiguous() for t in cache])
    check_attention(q, small, table - top, [400], out, lse, 1 / math.sqrt(d), False)


# ---------------------------------------------------------------- streams, graphs, the three together
def test_streams_and_concurrent_calls(fa):
    rng = np.random.default_rng(28)
    lens, page, d = [900, 20], 16, 64
    table, n_pages = random_table(rng, lens, page)
    cache = filled(fa, rng, "e4m3", n_pages, 2, page, d)
    tab, ln = ints(table.tolist()), ints(lens)
    qs = [torch.from_numpy(rng.standard_normal((2, 4, 2, d))).half().to(DEV) for _ in range(6)]
    want = [fa.attention_kvq8(q, cache, tab, ln, causal=True, n_parts=9) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [fa.attention_kvq8(q, cache, tab, ln, causal=True, n_parts=9,
                             stream=streams[i % 3] if i < 3 else streams[i % 3].cuda_stream)
           for i, q in enumerate(qs)]
    torch.cuda.synchronize()
    for (a, b), (c, e) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, e)
    status_ok(fa)


def test_decoding_loop_in_a_graph(fa):
    """A captured step (append, then attention) replayed while the lengths and inputs it reads move on; two graphs
    with their own workspaces replayed in turn."""
    rng = np.random.default_rng(29)
    page, d, H, Hkv, B = 16, 128, 4, 2, 3
    lens = [0, 15, 40]
    table, n_pages = random_table(rng, [n + 24 for n in lens], page)
    cache = fa.kv_cache_q8(n_pages, Hkv, page, d, torch.float8_e4m3fn, DEV)
    start = torch.from_numpy(rng.standard_normal((sum(lens), Hkv, d))).bfloat16().to(DEV)
    tab, cu1 = ints(table.clip(max=n_pages - 1).tolist()), ints([0, 1, 2, 3])
    fa.kvq8_append(cache, start, start, tab, ints([0, 0, 15, 55]), ints([0, 0, 0]), 40)
    held, seen = ints(lens), ints([n + 1 for n in lens])
    k, v = (torch.zeros((B, Hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros((B, H, 1, d), dtype=torch.bfloat16, device=DEV)

    def step():
        fa.kvq8_append(cache, k, v, tab, cu1, held, 1)
        got = fa.attention_kvq8(q, cache, tab, seen, n_parts=2)
        held.add_(1)
        seen.add_(1)
        return got

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        graphs.append((g, res))
    for i in range(20):
        k.copy_(torch.from_numpy(rng.standard_normal((B, Hkv, d))).bfloat16())
        v.copy_(torch.from_numpy(rng.standard_normal((B, Hkv, d))).bfloat16() * 2 ** (i // 7))
        q.copy_(torch.from_numpy(rng.standard_normal((B, H, 1, d))).bfloat16())
        g, (out, lse) = graphs[i % 2]
        g.replay()
        status_ok(fa)
        check_attention(q, cache, table, [n + i + 1 for n in lens], out, lse, 1 / math.sqrt(d), False)


def test_prompt_then_steps_then_packed_forward(fa):
    """Prompts written in one call, drafted tokens checked causally, and the cached prefix read back for the packed
    forward: the last rows of the packed forward are the decoding forward's."""
    rng = np.random.default_rng(30)
    page, d, H, Hkv = 32, 128, 8, 2
    lens = [70, 33, 200]
    table, n_pages = random_table(rng, lens, page)
    tab = ints(table.clip(max=n_pages - 1).tolist())
    cache = fa.kv_cache_q8(n_pages, Hkv, page, d, torch.int8, DEV)
    total = sum(lens)
    cu = [0] + [int(c) for c in np.cumsum(lens)]
    k, v = (torch.from_numpy(rng.standard_normal((total, Hkv, d))).bfloat16().to(DEV) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((total, H, d))).bfloat16().to(DEV)
    fa.kvq8_append(cache, k, v, tab, ints(cu), ints([0, 0, 0]), max(lens))
    kr, vr = fa.kvq8_read(cache, tab, ints(cu), total, max(lens))
    packed, plse = fa.attention_varlen(q, kr, vr, ints(cu), max(lens), causal=True)
    Nq = 4
    last = torch.stack([q[cu[s + 1] - Nq : cu[s + 1]].transpose(0, 1) for s in range(3)]).contiguous()
    out, lse = fa.attention_kvq8(last, cache, tab, ints(lens), causal=True)
    status_ok(fa)
    check_attention(last, cache, table, lens, out, lse, 1 / math.sqrt(d), True)
    for s in range(3):
        rows = packed[cu[s + 1] - Nq : cu[s + 1]].transpose(0, 1).float()
        # both rounded to bf16, the packed forward's weights too: 3 halves of a step of |o| <= ~1
        assert float((rows - out[s].float()).abs().max()) <= 2e-2
        assert float((plse[:, cu[s + 1] - Nq : cu[s + 1]] - lse[s]).abs().max()) <= 1e-3
