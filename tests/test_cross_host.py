"""The entry points for keys of another length refuse bad arguments on the host, before anything is launched. CPU only."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    return mod


def _args(ptrs):
    return [ctypes.c_void_p(x) if x else None for x in ptrs]


def fwd(fa, name="fa_fwd_cross", ptrs=None, lens=0, B=2, H=4, Hkv=2, Nq=5, Nk=300, d=64, n_splits=1, ws=0, ws_bytes=0):
    p = [0x10000 * (i + 1) for i in range(5)] if ptrs is None else ptrs
    q, k, v, out, lse = _args(p)
    return getattr(fa.lib, name)(q, k, v, ctypes.c_void_p(lens) if lens else None, out, lse, B, H, Hkv, Nq, Nk, d,
                                 ctypes.c_float(0.1), n_splits, ctypes.c_void_p(ws) if ws else None, ws_bytes, None)


def bwd(fa, name="fa_bwd_cross", ptrs=None, lens=0, B=2, H=4, Hkv=2, Nq=5, Nk=300, d=64, ws=0x900000, ws_bytes=1 << 30):
    p = [0x10000 * (i + 1) for i in range(9)] if ptrs is None else ptrs
    a = _args(p)
    return getattr(fa.lib, name)(*a[:3], ctypes.c_void_p(lens) if lens else None, *a[3:], B, H, Hkv, Nq, Nk, d,
                                 ctypes.c_float(0.1), ctypes.c_void_p(ws) if ws else None, ws_bytes, None)


@pytest.mark.parametrize("call,n,names", [(fwd, 5, ("fa_fwd_cross", "fa_fwd_cross_fp16")),
                                          (bwd, 9, ("fa_bwd_cross", "fa_bwd_cross_fp16"))])
def test_bad_arguments_are_refused(fa, call, n, names):
    for name in names:
        for i in range(n):
            p = [0x10000 * (j + 1) for j in range(n)]
            p[i] = 0
            assert call(fa, name, p) == fa.FA_ERR_NULL
            p[i] = 0x10000 * (i + 1) + 2
            assert call(fa, name, p) == fa.FA_ERR_ALIGN
        assert call(fa, name, lens=0x10002) == fa.FA_ERR_ALIGN
        for kw in (dict(B=0), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(Hkv=8), dict(Nq=0), dict(Nk=0),
                   dict(B=1 << 16, H=1 << 16), dict(B=1 << 14, H=64, Hkv=64, Nk=1 << 30)):
            assert call(fa, name, **kw) == fa.FA_ERR_SHAPE, kw
        for d in (32, 96, 256):
            assert call(fa, name, d=d) == fa.FA_ERR_UNSUPPORTED


def test_splits_and_workspaces_are_refused(fa):
    assert fwd(fa, n_splits=0) == fa.FA_ERR_SHAPE
    assert fwd(fa, n_splits=4) == fa.FA_ERR_SHAPE  # 300 keys are three blocks
    need = fa.fa_splitkv_workspace_bytes(2, 4, 5, 64, 3)
    assert fwd(fa, n_splits=3) == fa.FA_ERR_WORKSPACE
    assert fwd(fa, n_splits=3, ws=0x900010, ws_bytes=need) == fa.FA_ERR_WORKSPACE
    assert fwd(fa, n_splits=3, ws=0x900000, ws_bytes=need - 1) == fa.FA_ERR_WORKSPACE
    need = fa.fa_bwd_cross_workspace_bytes(2, 4, 2, 5, 300, 64)
    assert need >= fa.fa_bwd_workspace_bytes(2, 4, 5, 64)
    for bad in ((0, 4, 2, 5, 300, 64), (2, 4, 3, 5, 300, 64), (2, 4, 2, 5, 0, 64)):
        assert fa.lib.fa_bwd_cross_workspace_bytes(*bad) == fa.FA_ERR_SHAPE
    assert fa.lib.fa_bwd_cross_workspace_bytes(2, 4, 2, 5, 300, 96) == fa.FA_ERR_UNSUPPORTED
    assert bwd(fa, ws=0) == fa.FA_ERR_WORKSPACE
    assert bwd(fa, ws_bytes=need - 1) == fa.FA_ERR_WORKSPACE
    assert fa.lib.fa_cross_num_splits(0, 1, 1, 1) == fa.FA_ERR_SHAPE
    for B, H, Nq, Nk in ((1, 1, 1, 1), (1, 8, 40, 1500), (2, 4, 300, 100000), (100, 64, 7, 5000)):
        assert 1 <= fa.fa_cross_num_splits(B, H, Nq, Nk) <= (Nk + 127) // 128


def test_binding_refuses(fa):
    q, k = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 7, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 3)
    with pytest.raises(ValueError):
        fa.attention_cross(q, k, k, n_splits=1)  # CPU tensors
    with pytest.raises(ValueError):
        fa.attention_cross(q.float(), k.float(), k.float())
    with pytest.raises(ValueError):
        fa.attention_cross_backward(q, k, k, q, q, lse)
