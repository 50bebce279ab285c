"""A NaN in a query makes its own row NaN, out and lse, in every forward, and no other row's bits change; only a row that
sees no key is 0 and -inf."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def randn(seed, dtype, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).to(DEV)


def check(fa, call, q, at, lse_at=None):
    """call(q) -> out, lse; `at` the index of the row in q and out, `lse_at` in lse."""
    lse_at = at if lse_at is None else lse_at
    want, wl = call(q)
    bad = q.clone()
    bad[at + (3,)] = float("nan")
    out, lse = call(bad)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK
    assert bool(torch.isnan(out[at]).all()) and bool(torch.isnan(lse[lse_at]))
    out[at], lse[lse_at] = want[at], wl[lse_at]
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Nq,Nk,n_splits", [(1, 700, 1), (1, 2000, 5), (5, 700, 1), (16, 900, 4), (6, 3, 1)])
def test_decoding(fa, dtype, d, causal, Nq, Nk, n_splits):
    q, k, v = (randn(i, dtype, 2, 2, n, d) for i, n in enumerate((Nq, Nk, Nk)))
    check(fa, lambda x: fa.attention_decode(x, k, v, causal=causal, n_splits=n_splits), q, (1, 0, Nq - 1))
    if dtype == "bf16":
        def noalloc(x):
            out, lse = torch.empty_like(x), torch.empty(x.shape[:3], device=DEV)
            fa.fa_fwd_splitkv_noalloc(x, k, v, out, lse, 0.1, causal, n_splits)
            return out, lse

        check(fa, noalloc, q, (0, 1, Nq - 1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("causal", [False, True])
def test_forwards(fa, dtype, d, causal):
    N = 300
    q, k, v = (randn(i, dtype, 1, 2, N, d) for i in range(3))
    check(fa, lambda x: fa.attention(x, k, v, causal=causal), q, (0, 1, 217))
    check(fa, lambda x: fa.attention(x, k, v, scale=-0.1, causal=causal), q, (0, 0, 17))  # (scores scaled one by one)
    mask = torch.zeros(1, N, N, device=DEV)
    mask[:, :, 250:] = -float("inf")
    mask[:, 5] = -float("inf")
    check(fa, lambda x: fa.attention(x, k, v, mask, causal=causal), q, (0, 0, 131))
    if dtype == "fp32":
        return
    mask[:, :, :250] = 0.25
    check(fa, lambda x: fa.attention(x, k, v, mask, causal=causal), q, (0, 1, 131))  # no 0 / -inf mask
    check(fa, lambda x: fa.attention_bias(x, k, v, mask[:, None].expand(1, 2, N, N).contiguous(), causal=causal), q, (0, 1, 9))
    check(fa, lambda x: fa.attention_dropout(x, k, v, 0.25, 7, causal=causal), q, (0, 0, 299))
    qt, kt, vt = (t[0].transpose(0, 1).contiguous() for t in (q, k, v))
    cu = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device=DEV)
    check(fa, lambda x: fa.attention_varlen(x, kt, vt, cu, 200, causal=causal), qt, (120, 1), (1, 120))


@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_key_reaches_the_rows_that_see_it(fa, d):
    q, k, v = (randn(i, "bf16", 1, 2, n, d) for i, n in enumerate((4, 500, 500)))
    want, wl = fa.attention_decode(q, k, v, n_splits=3)
    k[0, 1, 498, 5] = float("nan")
    for n_splits in (1, 3):
        out, lse = fa.attention_decode(q, k, v, causal=True, n_splits=n_splits)  # row 2 and row 3 see key 498
        assert bool(torch.isnan(out[0, 1, 2:]).all()) and bool(torch.isnan(lse[0, 1, 2:]).all())
        assert not bool(torch.isnan(out[0, 0]).any()) and not bool(torch.isnan(out[0, 1, :2]).any())
    one, ol = fa.attention_decode(q[:, :, :1].contiguous(), k, v, n_splits=2)
    assert bool(torch.isnan(one[0, 1]).all()) and bool(torch.isnan(ol[0, 1]).all())
    assert not bool(torch.isnan(one[0, 0]).any()) and bool(torch.isfinite(ol[0, 0]).all())
