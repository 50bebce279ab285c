"""GPU: small softmax weights of large values behind a shared prefix, where pages' V scales lie 2^3 to 2^24 apart: every way
of doing the prefix gives what the attention over the whole gives.

Tolerance: the softmax weights are rounded to fp16 relative to the row's largest contribution p_j vs_j (vs the V scale of
key j's page), 2^-11 of themselves or 2^-25 of that largest one, times the code, at most cmax. The rest as in test_gpu_kvq8:
    |o - ref| <= (2^-11 + 2^-12) sum_j p_j |v_j| + 2^-25 n cmax max_j(p_j vs_j) + half_step |ref| + tiny
with p_j = exp(s_j) / sum exp(s). (The output's rounding is off by half a step, and a step is never less than the type's
smallest subnormal number: half of that, tiny, is 2^-25 for fp16, which outputs of V scales near 2^-28 meet, and 2^-134 for bf16.)"""
import math

import numpy as np
import pytest
import torch

import kvq8_ref as ref
from test_gpu_kvq8 import CODE, DEV, DT, as_ref, filled, ints, random_table, status_ok

pytestmark = pytest.mark.gpu
SPLITS = [None, (0, 0), (0, 7), (1, 0), (2, 3), (5, 0)]  # (n_splits, n_parts)


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def check(fa, q, cache, shared, prefix, table, lens, scale, page):
    kc, ks, vc, vs = as_ref(cache)
    half, tiny = (2.0 ** -8, 2.0 ** -134) if q.dtype == torch.bfloat16 else (2.0 ** -11, 2.0 ** -25)
    cmax = np.abs(vc).max()
    qn = q.cpu().double().numpy()
    want, tol, lse = [], [], []
    for b, n in enumerate(lens):
        k, v = (np.concatenate([ref.gather(c, s, shared, prefix), ref.gather(c, s, table[b], n)], 1)
                for c, s in ((kc, ks), (vc, vs)))
        rows = np.concatenate([np.asarray(shared)[np.arange(prefix) // page], np.asarray(table[b])[np.arange(n) // page]])
        v_scale = vs[rows.astype(int)].T  # [Hkv, keys]
        o, l, mag, _, _ = ref.attend(qn[b], k, v, scale, False)
        group = qn.shape[1] // k.shape[0]
        s = scale * np.einsum("hqd,hjd->hqj", qn[b], np.repeat(k, group, 0))
        largest = (np.exp(s - l[..., None]) * np.repeat(v_scale, group, 0)[:, None]).max(-1)
        want.append(o)
        lse.append(l)
        tol.append((2.0 ** -11 + 2.0 ** -12) * mag + 2.0 ** -25 * k.shape[1] * cmax * largest[..., None] + half * np.abs(o) + tiny)
    worst = {}
    for splits in SPLITS:
        kw = {}
        if splits is not None:
            kw.update(n_splits=min(splits[0], (prefix + 127) // 128), n_parts=splits[1])
        out, got = fa.attention_kvq8_prefix(q, cache, ints([int(x) for x in shared]), ints([prefix]), ints(table.tolist()),
                                            ints(lens), scale=scale, **kw)
        status_ok(fa)
        o, l = out.cpu().double().numpy(), got.cpu().double().numpy()
        worst[splits] = max(float((np.abs(o[b] - want[b]) / tol[b]).max()) for b in range(len(lens)))
        for b in range(len(lens)):
            assert np.all(np.abs(l[b] - lse[b]) <= 2.0 ** -13 + 2.0 ** -22 * np.abs(lse[b])), splits
    assert max(worst.values()) <= 1.0, worst


@pytest.mark.parametrize("sink", ["first", "last", "middle"])
@pytest.mark.parametrize("fmt,dtype,d", [("int8", "fp16", 64), ("e4m3", "bf16", 128)])
@pytest.mark.parametrize("apart", [3, 7, 8, 19, 20, 24])
def test_a_sink_of_small_values(fa, apart, fmt, dtype, d, sink):
    """One page of weight 1 and small values, 2500 keys of weights 2^-22 to 2^-26 under a V scale 2^apart times its own. The
    second head's queries are so small that its weights are equal, and the third's half of the first's."""
    rng = np.random.default_rng(apart)
    page, prefix, lens, H = 16, 2500, [33, 0], 3
    t, n_pages = random_table(rng, [prefix, *lens], page)
    shared, table = t[0], t[1:, :3]
    cache = filled(fa, rng, fmt, n_pages, 1, page, d)
    k = np.zeros((n_pages, 1, page, d))
    k[..., 0] = -rng.choice([52.0, 56.0, 60.0, 64.0], k.shape[:3])
    at = shared[{"first": 0, "last": len(shared) - 2, "middle": len(shared) // 2}[sink]]
    k[at, ..., 0] = 0.0
    cache.k_codes.copy_(torch.from_numpy(k).to(CODE[fmt]).to(DEV))
    cache.k_scale.fill_(0.25)
    cache.v_scale.fill_(2.0 ** -4)
    cache.v_scale[at] = 2.0 ** (-4 - apart)
    x = torch.zeros((2, H, 1, d))
    x[:, 0, :, 0], x[:, 1, :, 0], x[:, 2, :, 0] = 1.0, 2.0 ** -120 if dtype == "bf16" else 2.0 ** -24, 0.5
    check(fa, x.to(DT[dtype]).to(DEV), cache, shared, prefix, table, lens, 26 * math.log(2) / 16, page)


@pytest.mark.parametrize("fmt,d", [("int8", 128), ("e4m3", 64)])
@pytest.mark.parametrize("apart", [6, 7, 8, 12])
def test_a_sink_before_a_long_document(fa, apart, fmt, d):
    """The same with 30000 keys of weights near 2^-24.5 and values of one sign, whose losses would add up."""
    rng = np.random.default_rng(50 + apart)
    page, prefix, H = 128, 30000, 2
    t, n_pages = random_table(rng, [prefix, 0], page)
    shared, table = t[0], t[1:, :1]
    cache = filled(fa, rng, fmt, n_pages, 1, page, d)
    k = np.zeros((n_pages, 1, page, d))
    k[..., 0] = -rng.choice([60.0, 64.0], k.shape[:3])
    k[shared[0], ..., 0] = 0.0
    cache.k_codes.copy_(torch.from_numpy(k).to(CODE[fmt]).to(DEV))
    cache.v_codes.copy_(torch.from_numpy(rng.integers(10, 16, k.shape).astype(np.float64)).to(CODE[fmt]).to(DEV))
    cache.k_scale.fill_(0.25)
    cache.v_scale.fill_(2.0 ** -4)
    cache.v_scale[shared[0]] = 2.0 ** (-4 - apart)
    x = torch.zeros((1, H, 1, d))
    x[..., 0] = 1.0
    check(fa, x.half().to(DEV), cache, shared, prefix, table, [0], 25.3 * math.log(2) / 16, page)


@pytest.mark.parametrize("fmt,dtype,d", [("int8", "bf16", 128), ("e4m3", "fp16", 64)])
@pytest.mark.parametrize("apart", [3, 7, 8, 20])
def test_scales_against_scores(fa, apart, fmt, dtype, d):
    """Random keys and values whose pages' V scales fall as the pages' scores rise, so that small weights and large values
    are everywhere the same order; many rows, some of them behind keys of their own."""
    rng = np.random.default_rng(100 + apart)
    page, prefix, lens, H = 32, 1500, [int(x) for x in rng.integers(0, 60, 9)], 8
    t, n_pages = random_table(rng, [prefix, *lens], page)
    shared, table = t[0], t[1:, :2]
    cache = filled(fa, rng, fmt, n_pages, 2, page, d)
    k = ref.round_code(rng.standard_normal((n_pages, 2, page, d)) * 8, fmt)
    rank = rng.permutation(n_pages)[:, None, None] / n_pages  # of each page: 0 to 1
    k[..., 0] = np.round(64 * rank)
    cache.k_codes.copy_(torch.from_numpy(k).to(CODE[fmt]).to(DEV))
    cache.k_scale.fill_(2.0 ** -4)
    e = -4 - np.round(apart * rank[:, :, 0])
    cache.v_scale.copy_(torch.from_numpy(2.0 ** np.broadcast_to(e, (n_pages, 2))).float().to(DEV))
    x = rng.standard_normal((len(lens), H, 1, d)) * 0.2
    x[..., 0] = 4 * math.sqrt(d) * math.log(2) * apart / 16 * rng.choice([0.5, 1.0, 1.3], x.shape[:3])
    check(fa, torch.from_numpy(x).to(DT[dtype]).to(DEV), cache, shared, prefix, table, lens, 1 / math.sqrt(d), page)
