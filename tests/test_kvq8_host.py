"""The 8-bit cache's entry points refuse bad arguments on the host, before anything is launched; the reference that
the GPU tests compare with, against plain facts. CPU only."""
import ctypes

import numpy as np
import pytest
import torch

import kvq8_ref as ref


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    return mod


def P(i):
    return ctypes.c_void_p(0x10000 * i) if i else None


CACHE = dict(n_pages=10, max_pages=4, page=16, Hkv=2, d=64, format=0)


def append(fa, ptrs=None, strides=(128, 64, 128, 64), nseq=2, total=5, max_new=4, name="fa_kvq8_append", **kw):
    c = {**CACHE, **kw}
    p = [0x10000 * (i + 1) for i in range(9)] if ptrs is None else ptrs
    p = [ctypes.c_void_p(x) if x else None for x in p]
    return getattr(fa.lib, name)(p[0], p[1], *strides, p[2], p[3], nseq, total, max_new, p[4], p[5], p[6], p[7], p[8],
                                 c["n_pages"], c["max_pages"], c["page"], c["Hkv"], c["d"], c["format"], None)


def read(fa, ptrs=None, first=None, nseq=2, total=5, max_len=4, name="fa_kvq8_read", **kw):
    c = {**CACHE, **kw}
    p = [0x10000 * (i + 1) for i in range(8)] if ptrs is None else ptrs
    p = [ctypes.c_void_p(x) if x else None for x in p]
    return getattr(fa.lib, name)(*p[:5], c["n_pages"], c["max_pages"], c["page"], p[5],
                                 ctypes.c_void_p(first) if first else None, nseq, total, max_len, p[6], p[7], c["Hkv"],
                                 c["d"], c["format"], None)


def attend(fa, ptrs=None, B=2, H=4, Nq=1, max_len=64, n_parts=1, ws=0x100000, ws_bytes=1 << 20, name="fa_fwd_kvq8", **kw):
    c = {**CACHE, **kw}
    p = [0x10000 * (i + 1) for i in range(9)] if ptrs is None else ptrs
    p = [ctypes.c_void_p(x) if x else None for x in p]
    return getattr(fa.lib, name)(*p[:6], c["n_pages"], c["max_pages"], c["page"], p[6], p[7], p[8], B, H, c["Hkv"], Nq,
                                 max_len, c["d"], c["format"], ctypes.c_float(0.1), 0, n_parts,
                                 ctypes.c_void_p(ws) if ws else None, ws_bytes, None)


@pytest.mark.parametrize("call,n,names", [
    (append, 9, ("fa_kvq8_append", "fa_kvq8_append_fp16")),
    (read, 8, ("fa_kvq8_read", "fa_kvq8_read_fp16")),
    (attend, 9, ("fa_fwd_kvq8", "fa_fwd_kvq8_fp16")),
])
def test_cache_arguments_are_refused(fa, call, n, names):
    for name in names:
        for i in range(n):
            p = [0x10000 * (j + 1) for j in range(n)]
            p[i] = 0
            assert call(fa, p, name=name) == fa.FA_ERR_NULL
            p[i] = 0x10000 * (i + 1) + 2
            assert call(fa, p, name=name) == fa.FA_ERR_ALIGN
        for kw in (dict(n_pages=0), dict(max_pages=0), dict(Hkv=0), dict(max_pages=1 << 30)):
            assert call(fa, name=name, **kw) == fa.FA_ERR_SHAPE, kw
        for kw in (dict(page=8), dict(page=48), dict(page=256), dict(d=96), dict(d=256)):
            assert call(fa, name=name, **kw) == fa.FA_ERR_UNSUPPORTED, kw
        for kw in (dict(format=2), dict(format=-1)):
            assert call(fa, name=name, **kw) == fa.FA_ERR_ARG, kw


def test_append_and_read_sizes_are_refused(fa):
    for kw in (dict(nseq=0), dict(total=0), dict(max_new=0)):
        assert append(fa, **kw) == fa.FA_ERR_SHAPE
    for i in range(4):
        s = [128, 64, 128, 64]
        s[i] += 4
        assert append(fa, strides=s) == fa.FA_ERR_SHAPE
    for kw in (dict(nseq=0), dict(total=0), dict(max_len=0)):
        assert read(fa, **kw) == fa.FA_ERR_SHAPE
    assert read(fa, first=0x10002) == fa.FA_ERR_ALIGN


def test_attention_sizes_and_workspace_are_refused(fa):
    for kw in (dict(B=0), dict(H=0), dict(H=3), dict(Nq=0), dict(Nq=17), dict(max_len=0), dict(max_len=65),
               dict(n_parts=-1), dict(n_parts=(1 << 20) + 1), dict(B=1 << 20, H=1 << 12),
               dict(B=1 << 18, max_pages=1 << 14, max_len=1 << 18)):
        assert attend(fa, **kw) == fa.FA_ERR_SHAPE, kw
    need = fa.fa_kvq8_workspace_bytes(4, 2, 1, 64, 2)
    assert attend(fa, n_parts=2, ws=0) == fa.FA_ERR_WORKSPACE
    assert attend(fa, n_parts=2, ws=0x100010, ws_bytes=need) == fa.FA_ERR_WORKSPACE
    assert attend(fa, n_parts=2, ws_bytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert fa.lib.fa_kvq8_num_parts(1, 4, 3, 1, 100, 64) == fa.FA_ERR_SHAPE
    assert fa.lib.fa_kvq8_num_parts(1, 4, 2, 1, 100, 80) == fa.FA_ERR_UNSUPPORTED
    assert fa.lib.fa_kvq8_workspace_bytes(4, 3, 1, 64, 1) == fa.FA_ERR_SHAPE
    assert fa.lib.fa_kvq8_workspace_bytes(4, 2, 1, 96, 1) == fa.FA_ERR_UNSUPPORTED
    for B, Hkv, n in ((1, 1, 1), (1, 8, 100000), (300, 8, 5000), (4, 2, 63)):
        s = fa.fa_kvq8_num_parts(B, 4 * Hkv, Hkv, 1, n, 128)
        assert (s == 0) == (n <= 512) and s <= B * Hkv * ((n + 63) // 64)


def test_binding_refuses(fa):
    codes = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    scale = torch.zeros(4, 2)
    cache = fa.KVCacheQ8(codes, codes, scale, scale)
    table, cu, lens = (torch.zeros(s, dtype=torch.int32) for s in ((1, 4), (2,), (1,)))
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.kvq8_append(cache, x, x, table, cu, lens, 3)  # CPU tensors
    with pytest.raises(ValueError):
        fa.kvq8_read(cache, table, cu, 3, 3)
    with pytest.raises(ValueError):
        fa.attention_kvq8(torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16), cache, table, lens, n_parts=1)
    with pytest.raises(ValueError):
        fa.attention_kvq8(torch.zeros(1, 2, 1, 64), cache, table, lens)  # fp32 queries
    with pytest.raises(ValueError):
        fa.kv_cache_q8(4, 2, 16, 64, torch.uint8, "cpu")
    bad = fa.KVCacheQ8(codes.view(torch.uint8), codes, scale, scale)
    with pytest.raises(ValueError):
        fa.kvq8_read(bad, table, cu, 3, 3)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_reference_codes(fmt):
    """Every code rounds to itself, halfway values to even, and the scale is the smallest that holds the value."""
    if fmt == "e4m3":
        codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        codes = np.unique(codes[np.isfinite(codes)])
        x = np.random.default_rng(0).standard_normal(20000) * 100
        assert np.array_equal(ref.round_code(x, fmt), torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy())
    else:
        codes = np.arange(-127.0, 128.0)
        assert np.array_equal(ref.round_code(np.array([0.5, 1.5, -2.5, 300.0]), fmt), [0, 2, -2, 127])
    assert np.array_equal(ref.round_code(codes, fmt), codes)
    for a in (1.0, 126.99, 127.0, 127.01, 447.0, 448.0, 450.0, 2.0 ** -40 * 1.3):
        s = ref.scale_for(a, fmt)
        assert a <= ref.QMAX[fmt] * s and a > ref.QMAX[fmt] * s / 2
    assert ref.scale_for(0.0, fmt) == 0.0


def test_reference_attention_is_the_oracle(oracle_lib):
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 3, 64)), rng.standard_normal((2, 50, 64)), rng.standard_normal((2, 50, 64))
    out, lse, mag, _, _ = ref.attend(q, k, v, 0.125, False)
    want, wl = oracle_lib.attention(q[None], np.repeat(k, 2, 0)[None], np.repeat(v, 2, 0)[None], scale=0.125)
    assert np.allclose(out, want[0], atol=1e-12) and np.allclose(lse, wl[0], atol=1e-12)
    assert np.all(mag >= np.abs(out) - 1e-12)
    out, lse, *_ = ref.attend(q, k[:, :2], v[:, :2], 0.125, True)  # two keys, three rows: the first sees none
    assert np.all(out[:, 0] == 0) and np.all(np.isneginf(lse[:, 0])) and np.all(np.isfinite(lse[:, 1:]))
