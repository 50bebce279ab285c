"""Attention behind a shared prefix refuses bad arguments on the host, before anything is launched. CPU only."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    return mod


def attend(fa, ptrs=None, name="fa_fwd_kvq8_prefix", prefix_pages=5, n_pages=10, max_pages=4, page=16, B=2, H=4, Hkv=2, Nq=1,
           max_prefix=70, max_len=64, d=64, format=0, n_splits=0, n_parts=1, ws=0x10000000, ws_bytes=1 << 24):
    p = [0x100000 * (i + 1) for i in range(11)] if ptrs is None else ptrs
    p = [ctypes.c_void_p(x) if x else None for x in p]
    return getattr(fa.lib, name)(*p[:6], prefix_pages, p[6], p[7], n_pages, max_pages, page, p[8], p[9], p[10], B, H, Hkv, Nq,
                                 max_prefix, max_len, d, format, ctypes.c_float(0.1), 0, n_splits, n_parts,
                                 ctypes.c_void_p(ws) if ws else None, ws_bytes, None)


@pytest.mark.parametrize("name", ["fa_fwd_kvq8_prefix", "fa_fwd_kvq8_prefix_fp16"])
def test_arguments_are_refused(fa, name):
    for i in range(11):
        p = [0x100000 * (j + 1) for j in range(11)]
        p[i] = 0
        assert attend(fa, p, name=name) == fa.FA_ERR_NULL, i
        p[i] = 0x100000 * (i + 1) + 2
        assert attend(fa, p, name=name) == fa.FA_ERR_ALIGN, i
    for kw in (dict(n_pages=0), dict(max_pages=0), dict(Hkv=0), dict(B=0), dict(H=3), dict(Nq=0), dict(Nq=17), dict(max_len=0),
               dict(max_len=65), dict(max_prefix=0), dict(max_prefix=81), dict(prefix_pages=0), dict(n_parts=-1), dict(n_splits=-1),
               dict(n_splits=2), dict(max_prefix=1 << 30, prefix_pages=1 << 26), dict(max_prefix=2 ** 31 - 1, prefix_pages=1 << 28),
               dict(B=1 << 18, max_prefix=1 << 18, prefix_pages=1 << 14)):
        assert attend(fa, name=name, **kw) == fa.FA_ERR_SHAPE, kw
    for kw in (dict(page=8), dict(page=256), dict(d=96)):
        assert attend(fa, name=name, **kw) == fa.FA_ERR_UNSUPPORTED, kw
    assert attend(fa, name=name, format=2) == fa.FA_ERR_ARG


def test_workspace_is_refused(fa):
    for splits, parts in ((0, 1), (0, 3), (1, 0), (1, 2)):
        need = fa.fa_kvq8_prefix_workspace_bytes(2, 4, 2, 1, 70, 64, splits, parts)
        kw = dict(n_splits=splits, n_parts=parts)
        assert need > 0
        assert attend(fa, ws=0, **kw) == fa.FA_ERR_WORKSPACE
        assert attend(fa, ws=0x10000010, ws_bytes=need, **kw) == fa.FA_ERR_WORKSPACE
        assert attend(fa, ws_bytes=need - 1, **kw) == fa.FA_ERR_WORKSPACE
    assert fa.fa_kvq8_prefix_workspace_bytes(2, 4, 2, 1, 70, 64, 0, 0) == 0


def test_sizes_are_refused(fa):
    for args in ((0, 4, 2, 1, 10, 10, 64), (1, 4, 3, 1, 10, 10, 64), (1, 4, 2, 17, 10, 10, 64), (1, 4, 2, 1, 0, 10, 64),
                 (1, 4, 2, 1, 10, 0, 64), (1, 4, 2, 1, 1 << 30, 1, 64), (1 << 20, 1 << 12, 1, 1, 10, 10, 64), (1, 4, 2, 1, 10, 10, 80)):
        with pytest.raises(fa.FAError):
            fa.fa_kvq8_prefix_plan(*args)
    for args in ((0, 4, 2, 1, 10, 64, 0, 0), (1, 4, 3, 1, 10, 64, 0, 0), (1, 4, 2, 1, 10, 64, 2, 0), (1, 4, 2, 1, 10, 64, -1, 0),
                 (1, 4, 2, 1, 10, 64, 0, -1), (1, 4, 2, 1, 0, 64, 0, 0), (1, 4, 2, 1, 10, 72, 0, 0),
                 (1, 4, 2, 1, 1 << 30, 64, 4097, 0)):
        with pytest.raises(fa.FAError):
            fa.fa_kvq8_prefix_workspace_bytes(*args)
    for B, Hkv, G, prefix, n, d in ((1, 1, 1, 1, 1, 64), (64, 8, 8, 32768, 2048, 128), (3, 8, 1, 1000, 100, 64), (300, 2, 4, 100, 9, 128)):
        splits, parts = fa.fa_kvq8_prefix_plan(B, Hkv * G, Hkv, 1, prefix, n, d)
        assert 0 <= splits <= (prefix + 127) // 128 and parts >= 0
        assert fa.fa_kvq8_prefix_workspace_bytes(B, Hkv * G, Hkv, 1, prefix, d, splits, parts) >= 0


def test_binding_refuses(fa):
    codes, scale = torch.zeros(4, 2, 16, 64, dtype=torch.int8), torch.zeros(4, 2)
    cache = fa.KVCacheQ8(codes, codes, scale, scale)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    q = torch.zeros(1, 2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.attention_kvq8_prefix(q, cache, i32(3), i32(1), i32(1, 4), i32(1))  # CPU tensors
    with pytest.raises(ValueError):
        fa.attention_kvq8_prefix(q.float(), cache, i32(3), i32(1), i32(1, 4), i32(1))  # fp32 queries
