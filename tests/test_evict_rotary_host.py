"""Weights, eviction and rotary positions: refusals on the host, before anything is launched, and the references that
the GPU tests compare with, against plain facts. CPU only."""
import ctypes

import numpy as np
import pytest
import torch

import evict_ref as er
import kvq8_ref as ref


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    return mod


def pointers(n, given):
    p = [0x1000000 * (i + 1) for i in range(n)] if given is None else given
    return [ctypes.c_void_p(x) if x else None for x in p]


def weights(fa, ptrs=None, name="fa_kvq8_weights", n_pages=10, max_pages=4, page=16, B=2, H=4, Hkv=2, Nq=1, max_len=64, d=64,
            format=0):
    p = pointers(7, ptrs)
    return getattr(fa.lib, name)(*p[:4], n_pages, max_pages, page, *p[4:], B, H, Hkv, Nq, max_len, d, format,
                                 ctypes.c_float(0.1), 0, None)


def evict(fa, ptrs=None, n_pages=10, max_pages=4, page=16, keep=20, recent=3, nseq=2, Hkv=2, d=64, format=0, name=None):
    p = pointers(10, ptrs)
    return fa.lib.fa_kvq8_evict(*p[:5], n_pages, max_pages, page, p[5], p[6], keep, recent, *p[7:], nseq, Hkv, d, format, None)


@pytest.mark.parametrize("call,n,names", [(weights, 7, ("fa_kvq8_weights", "fa_kvq8_weights_fp16")), (evict, 10, ("fa_kvq8_evict",))])
def test_cache_arguments_are_refused(fa, call, n, names):
    for name in names:
        for i in range(n):
            p = [0x1000000 * (j + 1) for j in range(n)]
            p[i] = 0
            assert call(fa, p, name=name) == fa.FA_ERR_NULL
            p[i] = 0x1000000 * (i + 1) + 2
            assert call(fa, p, name=name) == fa.FA_ERR_ALIGN
        for kw in (dict(n_pages=0), dict(max_pages=0), dict(Hkv=0), dict(max_pages=1 << 30)):
            assert call(fa, name=name, **kw) == fa.FA_ERR_SHAPE, kw
        for kw in (dict(page=8), dict(page=48), dict(d=96), dict(d=256)):
            assert call(fa, name=name, **kw) == fa.FA_ERR_UNSUPPORTED, kw
        assert call(fa, name=name, format=2) == fa.FA_ERR_ARG


def test_weights_sizes_are_refused(fa):
    for kw in (dict(B=0), dict(H=0), dict(H=3), dict(Nq=0), dict(Nq=17), dict(max_len=0), dict(max_len=65), dict(B=1 << 20, H=1 << 12),
               dict(B=1 << 20, max_pages=1 << 16, max_len=1 << 20)):
        assert weights(fa, **kw) == fa.FA_ERR_SHAPE, kw


def test_evict_sizes_and_overlaps_are_refused(fa):
    for kw in (dict(keep=0), dict(keep=-1), dict(recent=-1), dict(recent=21), dict(keep=(1 << 30) + 1)):
        assert evict(fa, **kw) == fa.FA_ERR_ARG, kw
    for kw in (dict(nseq=0), dict(nseq=1 << 30)):
        assert evict(fa, **kw) == fa.FA_ERR_SHAPE, kw
    base = [0x1000000 * (i + 1) for i in range(10)]
    size = 2 * 2 * 64 * 4
    for i, j, off in ((9, 6, 0), (9, 6, size - 16), (6, 9, size - 16), (8, 6, 16), (8, 9, 16), (7, 5, 0), (7, 5, 4)):
        p = list(base)
        p[i] = p[j] + off  # weight_out on weight, kept on either, lens_out on kv_lens
        assert evict(fa, p) == fa.FA_ERR_ARG, (i, j, off)


@pytest.mark.parametrize("out", [7, 8, 9])
@pytest.mark.parametrize("other", range(10))
def test_evict_outputs_on_any_other_tensor_are_refused(fa, out, other):
    p = [0x1000000 * (i + 1) for i in range(10)]
    if out == other:
        return
    p[out] = p[other]
    assert evict(fa, p) == fa.FA_ERR_ARG


def rotary(fa, ptrs=None, strides=(0, 128, 64, 0, 128, 64), Hq=2, Hk=1, n_axes=2, inv=None, axis=None, pairs=32, B=1, N=3, d=64,
           name="fa_rotary"):
    p = pointers(5, ptrs)
    six = (ctypes.c_longlong * 6)(*strides)
    f = (ctypes.c_double * 64)(*(inv or [0.5] * 64))
    a = (ctypes.c_int * 64)(*(axis or [0, 1] * 32))
    return getattr(fa.lib, name)(p[0], p[1], six, Hq, p[2], p[3], six, Hk, p[4], n_axes, f, a, pairs, B, N, d, 0, None)


@pytest.mark.parametrize("name", ["fa_rotary", "fa_rotary_fp16"])
def test_rotary_arguments_are_refused(fa, name):
    for i in range(5):
        p = [0x1000000 * (j + 1) for j in range(5)]
        p[i] = 0
        assert rotary(fa, p, name=name) == fa.FA_ERR_NULL
        p[i] = 0x1000000 * (i + 1) + 2
        assert rotary(fa, p, name=name) == fa.FA_ERR_ALIGN
    for i in range(6):
        s = [0, 128, 64, 0, 128, 64]
        s[i] += 4
        assert rotary(fa, strides=s, name=name) == fa.FA_ERR_SHAPE
    for kw in (dict(Hq=0), dict(Hk=-1), dict(B=0), dict(N=0), dict(B=1 << 16, N=1 << 16), dict(pairs=0), dict(pairs=4), dict(pairs=12),
               dict(pairs=40)):
        assert rotary(fa, name=name, **kw) == fa.FA_ERR_SHAPE, kw
    assert rotary(fa, name=name, d=96) == fa.FA_ERR_UNSUPPORTED
    for kw in (dict(n_axes=0), dict(n_axes=9), dict(n_axes=1), dict(axis=[-1] * 64), dict(inv=[float("nan")] * 64),
               dict(inv=[float("inf")] * 64)):
        assert rotary(fa, name=name, **kw) == fa.FA_ERR_ARG, kw


@pytest.mark.parametrize("name", ["fa_rotary", "fa_rotary_fp16"])
def test_rotary_outputs_that_collide_are_refused(fa, name):
    base = [0x1000000 * (j + 1) for j in range(5)]
    # output rows on each other: a repeated token or head, half a row apart, tokens within the heads' reach, far out
    for s in ((0, 0, 64), (0, 128, 0), (0, 128, 32), (0, 64, 64), (0, 96, 64), (0, -128, 64), (0, 1 << 41, 64)):
        assert rotary(fa, strides=(0, 128, 64, *s), name=name) == fa.FA_ERR_SHAPE, s
    assert rotary(fa, strides=(384, 128, 64, 320, 128, 64), B=2, name=name) == fa.FA_ERR_SHAPE
    for i, j in ((0, 1), (2, 3)):  # in place, under other strides
        p = list(base)
        p[j] = p[i]
        assert rotary(fa, p, strides=(0, 128, 64, 0, 256, 64), name=name) == fa.FA_ERR_SHAPE
    for i, j in ((3, 1), (1, 2), (3, 0)):  # one output for both, q's on k, k's on q
        p = list(base)
        p[i] = p[j]
        assert rotary(fa, p, name=name) == fa.FA_ERR_ARG, (i, j)
    p = [base[0], base[0], base[0], base[0], base[4]]  # the same tensor for q and k, in place
    assert rotary(fa, p, Hq=1, name=name) == fa.FA_ERR_ARG


def test_bindings_refuse(fa):
    codes = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    scale = torch.zeros(4, 2)
    cache = fa.KVCacheQ8(codes, codes, scale, scale)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.kvq8_weights(q, cache, table, lens, torch.zeros(1, 2, 1), torch.zeros(1, 2, 64))  # CPU tensors
    with pytest.raises(ValueError):
        fa.kvq8_evict(cache, table, lens, torch.zeros(1, 2, 64), 10, 2)
    inv, axis = fa.rotary_frequencies(32, [8, 12, 12])
    with pytest.raises(ValueError):
        fa.rotary(torch.zeros(3, 2, 64), None, torch.zeros(3, 3, dtype=torch.int32), inv, axis)  # fp32
    with pytest.raises(ValueError):
        fa.rotary(q[0].transpose(0, 1), None, torch.zeros(3, 1, dtype=torch.int32), inv, axis)  # CPU
    for sections in ([8, 8], [40, -8], [8, 12, 13]):
        with pytest.raises(ValueError):
            fa.rotary_frequencies(32, sections)


def test_frequencies(fa):
    inv, axis = fa.rotary_frequencies(8, [2, 3, 3], theta=100.0)
    assert inv.tolist() == [100.0 ** (-i / 8) for i in range(8)] and axis.tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    _, axis = fa.rotary_frequencies(8, [2, 3, 3], interleaved=True)
    assert axis.tolist() == [0, 1, 2, 0, 1, 2, 1, 2]
    assert fa.rotary_frequencies(16)[1].tolist() == [0] * 16


def test_reference_choice():
    w = np.array([3.0, np.nan, 1.0, 3.0, -0.0, 0.0, 2.0, 9.0])
    assert er.keep_positions(w, 8, 2) == list(range(8))
    assert er.keep_positions(w, 2, 2) == [6, 7]
    assert er.keep_positions(w, 3, 2) == [1, 6, 7]
    assert er.keep_positions(w, 4, 2) == [0, 1, 6, 7]  # of equal ones the lower
    assert er.keep_positions(w, 6, 0) == [0, 1, 2, 3, 6, 7]
    assert er.keep_positions(w, 7, 0) == [0, 1, 2, 3, 4, 6, 7]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_reference_eviction_moves_values(fmt):
    """What is kept has its value, rounded to its new page's scale; pages without moves, and slots behind, stay."""
    rng = np.random.default_rng(0)
    codes = ref.round_code(rng.standard_normal((6, 2, 16, 8)) * 50, fmt)
    scales = 2.0 ** rng.integers(-3, 3, (6, 2))
    table, n = [4, 1, 5, 0], 60
    c, s = codes.copy(), scales.copy()
    w = rng.random((2, n))
    w[:, :16] = 5.0
    kept = [er.keep_positions(w[h], 40, 5) for h in range(2)]
    er.evict(c, s, fmt, [table], [n], [kept])
    was, now = ref.gather(codes, scales, table, n), ref.gather(c, s, table, 40)
    for h in range(2):
        top = np.abs(was[h][kept[h]]).reshape(40, -1).max(1)
        step = np.array([s[table[i // 16], h] for i in range(40)])[:, None] * (1 if fmt == "int8" else 32)
        assert np.all(np.abs(now[h] - was[h][kept[h]]) <= step / 2 + 1e-12) and top.max() > 0
    assert np.array_equal(c[4], codes[4]) and np.array_equal(c[0], codes[0]) and np.array_equal(c[5][:, 8:], codes[5][:, 8:])
    assert np.array_equal(c[[2, 3]], codes[[2, 3]])


def test_reference_weights_and_rotary():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((4, 2, 8)), rng.standard_normal((2, 30, 8))
    out, lse, *_ = ref.attend(q, k, k, 0.3, True)
    w, bound = er.weights(q, k, lse, 0.3, True)
    assert np.allclose(w.sum(-1), 4) and np.all(bound < 1e-3) and w[0, 29] > 0
    x = rng.standard_normal((5, 3, 16))
    pos = rng.integers(0, 100, (2, 5))
    inv, axis = np.array([1.0, 0.1, 0.01, 0.5]), [0, 1, 1, 0]
    y = er.rotary(x, pos, inv, axis, False)
    assert np.allclose(er.rotary(y, pos, inv, axis, True), x) and np.array_equal(y[..., 8:], x[..., 8:])
    z = (x[..., 1] + 1j * x[..., 5]) * np.exp(1j * pos[1][:, None] * 0.1)
    assert np.allclose(y[..., 1], z.real) and np.allclose(y[..., 5], z.imag)
