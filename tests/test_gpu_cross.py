"""GPU parity of the forward over keys of another length, and of its gradients, against plain 64-bit arithmetic.

Tolerances, per element, from the arithmetic (h: half a step of the 16-bit type relative to the value, 2^-8 or 2^-11;
e = 2^-12 covers fp32 sums, the exponentials and the error that lse's fp32 rounding gives a probability):
  out  (h + e) sum_j p_j |v_j| + h |out|                              (P rounded once, out rounded once)
  lse  2^-13 + 2^-22 |lse|
  dv   (h + e) sum_i p_ij |do_i| + h |dv|
  ds   s_ij = h |ds_ij| + p_ij h sum_t |do_it out_it| + e p_ij (|dp_ij| + |D_i|)      (dS rounded; D from the rounded out)
  dq   scale (sum_j s_ij |k_j| + e sum_j |ds_ij k_j|) + h |dq|,  dk the same over the queries of every head of the group
"""
import math

import numpy as np
import pytest
import torch

from cross_model import plan

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -12


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def status_ok(fa):
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_OK


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def inputs(seed, dtype, B, H, Hkv, Nq, Nk, d):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(B, H, Nq, d, generator=g).to(DT[dtype]).to(DEV)
    k, v = (torch.randn(B, Hkv, Nk, d, generator=g).to(DT[dtype]).to(DEV) for _ in range(2))
    do = torch.randn(B, H, Nq, d, generator=g).to(DT[dtype]).to(DEV)
    return q, k, v, do


def reference(q, k, v, lens, scale, do=None):
    """64-bit results and the bounds above: {"out", "lse"} or, with do, also {"dq", "dk", "dv"}; values (ref, tol)."""
    h = HALF[q.dtype]
    q, k, v = (t.cpu().double() for t in (q, k, v))
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    n = H // Hkv
    out, lse, t_out = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64), torch.zeros_like(q)
    if do is not None:
        do = do.cpu().double()
        dq, t_dq = torch.zeros_like(q), torch.zeros_like(q)
        dk, dv, t_dk, t_dv = (torch.zeros_like(k) for _ in range(4))
    for b in range(B):
        L = Nk if lens is None else lens[b]
        if L == 0:
            continue
        for i in range(H):
            kk, vv = k[b, i // n, :L], v[b, i // n, :L]
            s = scale * (q[b, i] @ kk.T)
            lse[b, i] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, i][:, None])
            out[b, i] = p @ vv
            t_out[b, i] = (h + E) * (p @ vv.abs()) + h * out[b, i].abs()
            if do is None:
                continue
            g = do[b, i]
            dp = g @ vv.T
            D = (p * dp).sum(-1, keepdim=True)
            ds = p * (dp - D)
            se = h * ds.abs() + p * h * (g.abs() * out[b, i].abs()).sum(-1, keepdim=True) + E * p * (dp.abs() + D.abs())
            dq[b, i] = scale * (ds @ kk)
            t_dq[b, i] = abs(scale) * (se @ kk.abs() + E * (ds.abs() @ kk.abs())) + h * dq[b, i].abs()
            dk[b, i // n, :L] += scale * (ds.T @ q[b, i])
            t_dk[b, i // n, :L] += abs(scale) * (se.T @ q[b, i].abs() + E * (ds.abs().T @ q[b, i].abs()))
            dv[b, i // n, :L] += p.T @ g
            t_dv[b, i // n, :L] += (h + E) * (p.T @ g.abs())
    r = {"out": (out, t_out), "lse": (lse, 2.0 ** -13 + 2.0 ** -22 * lse.abs())}
    if do is not None:
        r.update(dq=(dq, t_dq), dk=(dk, t_dk + h * dk.abs()), dv=(dv, t_dv + h * dv.abs()))
    return r


def check(name, got, ref):
    want, tol = ref
    got = got.cpu().double()
    seen = torch.isfinite(want)
    assert torch.equal(torch.isneginf(got), ~seen), name
    err = (got[seen] - want[seen]).abs()
    assert bool((err <= tol[seen] + 1e-30).all()), (name, float((err / (tol[seen] + 1e-30)).max()))


CASES = [
    # dtype, B, H, Hkv, Nq, Nk, d, lens
    ("bf16", 1, 1, 1, 1, 1, 64, None),
    ("fp16", 2, 2, 2, 35, 1500, 64, None),
    ("bf16", 3, 4, 2, 129, 300, 128, [300, 1, 0]),
    ("fp16", 4, 6, 2, 300, 130, 128, [129, 128, 127, 5]),
    ("bf16", 2, 8, 1, 257, 513, 64, [512, 400]),
    ("fp16", 5, 2, 1, 64, 200, 64, [0, 200, 16, 17, 113]),
    ("bf16", 1, 3, 3, 700, 90, 128, [33]),
    ("bf16", 2, 4, 4, 2, 2049, 128, [2049, 1025]),
    # more key blocks than SMs (one CTA for a block's gradients at d = 128, several blocks for a CTA at d = 64)
    ("bf16", 4, 8, 8, 130, 700, 64, [700, 641, 0, 130]),
    ("fp16", 4, 8, 8, 130, 700, 128, [700, 640, 129, 1]),
    ("fp16", 40, 10, 5, 3, 140, 64, [int(x) for x in np.random.default_rng(5).integers(0, 141, 40)]),
    ("bf16", 70, 4, 2, 130, 200, 64, [0] * 40 + [int(x) for x in np.random.default_rng(9).integers(0, 201, 30)]),
]


@pytest.mark.parametrize("dtype,B,H,Hkv,Nq,Nk,d,lens", CASES)
@pytest.mark.parametrize("n_splits", [None, 1, 2])
def test_forward(fa, dtype, B, H, Hkv, Nq, Nk, d, lens, n_splits):
    q, k, v, _ = inputs(Nq + Nk, dtype, B, H, Hkv, Nq, Nk, d)
    if n_splits is not None:
        n_splits = min(n_splits, (Nk + 127) // 128)
    out, lse = fa.attention_cross(q, k, v, None if lens is None else ints(lens), n_splits=n_splits)
    status_ok(fa)
    ref = reference(q, k, v, lens, 1 / math.sqrt(d))
    check("out", out, ref["out"])
    check("lse", lse, ref["lse"])


@pytest.mark.parametrize("dtype,B,H,Hkv,Nq,Nk,d,lens", CASES)
def test_gradients(fa, dtype, B, H, Hkv, Nq, Nk, d, lens):
    q, k, v, do = inputs(Nq + Nk, dtype, B, H, Hkv, Nq, Nk, d)
    kv_lens = None if lens is None else ints(lens)
    out, lse = fa.attention_cross(q, k, v, kv_lens)
    got = fa.attention_cross_backward(q, k, v, out, do, lse, kv_lens)
    status_ok(fa)
    ref = reference(q, k, v, lens, 1 / math.sqrt(d), do)
    for name, t in zip(("dq", "dk", "dv"), got):
        check(name, t, ref[name])


CUT = [
    # dtype, B, H, Hkv, Nq, Nk, d, lens: more key blocks than SMs, the last of them cut (8 of 160, 84 of 236, 16 of 168,
    # on 152 SMs; then 60 blocks, all cut)
    ("bf16", 4, 8, 4, 300, 1250, 128, [1250, 1250, 1249, 1153]),
    ("fp16", 4, 8, 4, 300, 1250, 64, None),
    ("fp16", 5, 8, 4, 1300, 1700, 128, [1700, 1600, 1664, 1281, 1000]),
    ("bf16", 6, 4, 2, 400, 1700, 64, None),
    ("fp16", 18, 6, 2, 257, 300, 64, [300, 0, 260, 1, 128, 129] * 3),
    ("bf16", 18, 6, 2, 257, 300, 128, [300, 0, 260, 1, 128, 129] * 3),
    ("fp16", 70, 4, 2, 130, 200, 128, [int(x) for x in np.random.default_rng(8).integers(0, 201, 70)]),  # many sequences
]


@pytest.mark.parametrize("dtype,B,H,Hkv,Nq,Nk,d,lens", CUT)
def test_gradients_of_cut_key_blocks(fa, dtype, B, H, Hkv, Nq, Nk, d, lens):
    """Key blocks whose queries are shared out over CTAs; dk and dv are the same bits every time."""
    valid = sum((n + 127) // 128 for n in ([Nk] * B if lens is None else lens)) * Hkv
    _, parts, _ = plan(valid, H // Hkv * ((Nq + 127) // 128), fa.fa_num_sms())
    if fa.fa_num_sms() == 152:
        assert parts > 1
    q, k, v, do = inputs(Nq + Nk, dtype, B, H, Hkv, Nq, Nk, d)
    kv_lens = None if lens is None else ints(lens)
    out, lse = fa.attention_cross(q, k, v, kv_lens)
    got = fa.attention_cross_backward(q, k, v, out, do, lse, kv_lens)
    again = fa.attention_cross_backward(q, k, v, out, do, lse, kv_lens)
    status_ok(fa)
    assert torch.equal(got[1], again[1]) and torch.equal(got[2], again[2])
    ref = reference(q, k, v, lens, 1 / math.sqrt(d), do)
    for name, t in zip(("dq", "dk", "dv"), got):
        check(name, t, ref[name])


def test_gradients_against_differences(fa):
    """d/dt of sum(do * out) along a random direction, by central differences of the 64-bit forward."""
    B, H, Hkv, Nq, Nk, d, lens = 2, 4, 2, 40, 150, 64, [150, 77]
    q, k, v, do = inputs(3, "fp16", B, H, Hkv, Nq, Nk, d)
    out, lse = fa.attention_cross(q, k, v, ints(lens))
    grads = fa.attention_cross_backward(q, k, v, out, do, lse, ints(lens))
    status_ok(fa)
    g = torch.Generator().manual_seed(9)
    base = [t.cpu().double() for t in (q, k, v)]
    w = do.cpu().double()

    def f(args):
        o = torch.zeros_like(args[0])
        for b in range(B):
            for i in range(H):
                kk, vv = args[1][b, i // 2, : lens[b]], args[2][b, i // 2, : lens[b]]
                o[b, i] = torch.softmax(args[0][b, i] @ kk.T / 8.0, -1) @ vv
        return float((o * w).sum())

    for n, grad in enumerate(grads):
        u = torch.randn(base[n].shape, generator=g, dtype=torch.float64)
        step = 1e-5
        up, down = ([b + s * u if m == n else b for m, b in enumerate(base)] for s in (step, -step))
        want = (f(up) - f(down)) / (2 * step)
        got = float((grad.cpu().double() * u).sum())
        # every element's error below 2^-8 of the gradients' norm, and of random sign against u: 6 sigma
        assert abs(got - want) <= 6 * 2.0 ** -8 * float(grad.double().norm()), (n, got, want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_what_lies_past_the_keys_does_not_matter(fa, dtype, d):
    """NaN, infinities and huge values in K and V past kv_lens change nothing, forward and backward."""
    B, H, Hkv, Nq, Nk = 4, 4, 2, 150, 400
    lens = [399, 129, 16, 0]
    q, k, v, do = inputs(11, dtype, B, H, Hkv, Nq, Nk, d)
    for b, n in enumerate(lens):
        k[b, :, n:] = 0
        v[b, :, n:] = 0
    clean = [fa.attention_cross(q, k, v, ints(lens), n_splits=s) for s in (1, 3)]
    grads = fa.attention_cross_backward(q, k, v, *[clean[0][0], do, clean[0][1]], ints(lens))
    for b, n in enumerate(lens):
        bad = torch.tensor([float("nan"), float("inf"), -float("inf"), 6e4], device=DEV).to(k.dtype)
        k[b, :, n:] = bad[torch.arange((Nk - n) * d, device=DEV) % 4].view(Nk - n, d)
        v[b, :, n:] = bad[torch.arange((Nk - n) * d, device=DEV) % 3].view(Nk - n, d)
    for s, (o, l) in zip((1, 3), clean):
        out, lse = fa.attention_cross(q, k, v, ints(lens), n_splits=s)
        assert torch.equal(out, o) and torch.equal(lse, l)
    got = fa.attention_cross_backward(q, k, v, clean[0][0], do, clean[0][1], ints(lens))
    status_ok(fa)
    for name, a, b in zip(("dq", "dk", "dv"), got, grads):
        assert bool(torch.isfinite(a).all()), name
        if name == "dq":  # accumulated in an order that varies
            assert bool(((a.double() - b.double()).abs() <= 2 * HALF[a.dtype] * b.double().abs() + 1e-4).all())
        else:
            assert torch.equal(a, b), name
    for b, n in enumerate(lens):
        assert bool((got[1][b, :, n:] == 0).all()) and bool((got[2][b, :, n:] == 0).all())
    assert bool((got[0][3] == 0).all()) and bool((clean[0][0][3] == 0).all())
    assert bool(torch.isneginf(clean[0][1][3]).all())


def test_lengths_out_of_range_count_as_zero(fa):
    q, k, v, do = inputs(12, "bf16", 3, 2, 1, 20, 140, 64)
    lens = ints([141, 100, -1])
    out, lse = fa.attention_cross(q, k, v, lens)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_SEQLENS
    dq, dk, dv = fa.attention_cross_backward(q, k, v, out, do, lse, lens)
    torch.cuda.synchronize()
    assert fa.fa_get_device_status() == fa.FA_ERR_SEQLENS
    ref = reference(q, k, v, [0, 100, 0], 1 / 8, do)
    for name, t in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, t, ref[name])
    status_ok(fa)


@pytest.mark.parametrize("n_splits", [1, 3])
def test_a_nan_query_stays_its_own_row(fa, n_splits):
    q, k, v, _ = inputs(19, "fp16", 2, 2, 1, 30, 400, 64)
    want, wl = fa.attention_cross(q, k, v, n_splits=n_splits)
    q[1, 0, 7, 3] = float("nan")
    out, lse = fa.attention_cross(q, k, v, n_splits=n_splits)
    status_ok(fa)
    assert bool(torch.isnan(out[1, 0, 7]).all()) and bool(torch.isnan(lse[1, 0, 7]))
    kept = torch.ones(lse.shape, dtype=torch.bool, device=DEV)
    kept[1, 0, 7] = False
    assert torch.equal(out[kept], want[kept]) and torch.equal(lse[kept], wl[kept])


def test_equal_lengths_are_the_plain_forward_bit_for_bit(fa):
    q, k, v, _ = inputs(13, "bf16", 2, 3, 3, 700, 700, 128)
    out, lse = fa.attention_cross(q, k, v, n_splits=1)
    want, wl = fa.attention(q, k, v)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    status_ok(fa)


def test_guard_bands(fa):
    """Nothing is written outside out, lse, dq, dk, dv and the workspaces."""
    B, H, Hkv, Nq, Nk, d, lens = 2, 4, 2, 77, 210, 64, [210, 130]
    q, k, v, do = inputs(14, "fp16", B, H, Hkv, Nq, Nk, d)

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * 4096,), 3.0, dtype=dtype, device=DEV)
        return buf, buf[4096 : 4096 + n].view(shape)

    bo, out = guarded(q.shape, q.dtype)
    bl, lse = guarded(q.shape[:3], torch.float32)
    nb = fa.fa_splitkv_workspace_bytes(B, H, Nq, d, 2)
    ws = torch.full((nb + 512,), 7, dtype=torch.uint8, device=DEV)
    fa.fa_fwd_cross_fp16(q, k, v, ints(lens), out, lse, 0.125, 2, ws[:nb])
    bq, dq = guarded(q.shape, q.dtype)
    bk, dk = guarded(k.shape, k.dtype)
    bv, dv = guarded(k.shape, k.dtype)
    nb2 = fa.fa_bwd_cross_workspace_bytes(B, H, Hkv, Nq, Nk, d)
    ws2 = torch.full((nb2 + 512,), 7, dtype=torch.uint8, device=DEV)
    fa.fa_bwd_cross_fp16(q, k, v, ints(lens), out, do, lse, dq, dk, dv, 0.125, ws2[:nb2])
    status_ok(fa)
    for b in (bo, bl, bq, bk, bv):
        assert bool((b[:4096] == 3.0).all()) and bool((b[-4096:] == 3.0).all())
    assert bool((ws[nb:] == 7).all()) and bool((ws2[nb2:] == 7).all())
    ref = reference(q, k, v, lens, 0.125, do)
    for name, t in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        check(name, t, ref[name])


def test_training_step_in_a_graph_and_streams(fa):
    """Forward and backward captured once, replayed on other inputs and lengths; and the same on another stream."""
    B, H, Hkv, Nq, Nk, d = 2, 4, 1, 50, 300, 128
    q, k, v, do = inputs(15, "bf16", B, H, Hkv, Nq, Nk, d)
    lens = ints([300, 300])

    def step(stream=None):
        out, lse = fa.attention_cross(q, k, v, lens, stream=stream)
        return (out, lse) + fa.attention_cross_backward(q, k, v, out, do, lse, lens, stream=stream)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = step()
    for seed, n in ((16, [300, 5]), (17, [131, 0])):
        for t, x in zip((q, k, v, do), inputs(seed, "bf16", B, H, Hkv, Nq, Nk, d)):
            t.copy_(x)
        lens.copy_(ints(n))
        g.replay()
        status_ok(fa)
        ref = reference(q, k, v, n, 1 / math.sqrt(d), do)
        for name, t in zip(("out", "lse", "dq", "dk", "dv"), res):
            check(name, t, ref[name])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = step(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(other[0], res[0]) and torch.equal(other[1], res[1])
    assert torch.equal(other[3], res[3]) and torch.equal(other[4], res[4])


def test_encoder_states_in_training_and_in_the_8_bit_cache(fa):
    """An encoder's keys and values quantised once into the cache: a decoder's tokens attend to them there as they do,
    within the codes' rounding, through the 16-bit forward."""
    B, H, Hkv, Nk, d = 3, 4, 2, 250, 64
    lens = [250, 100, 17]
    q, k, v, _ = inputs(18, "bf16", B, H, Hkv, 4, Nk, d)
    page = 32
    width = (Nk + page - 1) // page
    cache = fa.kv_cache_q8(B * width, Hkv, page, d, torch.int8, DEV)
    table = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    packed = [torch.cat([t[b, :, :n].transpose(0, 1) for b, n in enumerate(lens)]).contiguous() for t in (k, v)]
    cu = ints([0] + [int(x) for x in np.cumsum(lens)])
    fa.kvq8_append(cache, *packed, table, cu, ints([0] * B), max(lens))
    out, lse = fa.attention_kvq8(q, cache, table, ints(lens))
    kr, vr = fa.kvq8_read(cache, table, cu, sum(lens), max(lens))
    for b, n in enumerate(lens):
        k[b, :, :n] = kr[cu[b] : cu[b + 1]].transpose(0, 1)
        v[b, :, :n] = vr[cu[b] : cu[b + 1]].transpose(0, 1)
    want, wl = fa.attention_cross(q, k, v, ints(lens))
    status_ok(fa)
    ref = reference(q, k, v, lens, 1 / 8)  # int8 codes under powers of two are bf16 numbers: k, v are the cache's values
    check("out", want, ref["out"])
    check("out", out, ref["out"])
    check("lse", lse, ref["lse"])
    check("lse", wl, ref["lse"])
