"""GPU tests of the 8-bit cache's operators as a server uses them together: rotary positions, appending, attention behind
a shared prefix, the keys' weights and eviction; several calls at once; and caches whose offsets pass 32 bits. Against the
definitions in 64 bits (kvq8_ref, evict_ref) with the tolerances of each operator's own tests."""
import math

import numpy as np
import pytest
import torch

import evict_ref as er
import kvq8_ref as ref
from test_gpu_kvq8 import CODE, DEV, DT, as_ref, check_cache, filled, ints, random_table, status_ok
from test_gpu_kvq8_evict import make_weights
from test_gpu_kvq8_prefix import check, tables
from test_gpu_rotary import check as check_rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


@pytest.mark.parametrize("fmt,dtype,B,H,Hkv,Nq,d,page,prefix", [
    ("int8", "bf16", 4, 8, 2, 1, 128, 16, 333), ("e4m3", "fp16", 3, 6, 3, 3, 64, 32, 129), ("int8", "bf16", 40, 8, 1, 1, 64, 16, 700),
])
def test_serving_loop(fa, fmt, dtype, B, H, Hkv, Nq, d, page, prefix):
    """Steps of Nq new tokens each: turned, appended, attended to behind the prefix, weighed; at a budget, evicted."""
    rng = np.random.default_rng(prefix)
    budget, over, steps = 48, 24, 40 // Nq
    cap = (budget + over + Nq + page - 1) // page * page
    shared, table, n_pages = tables(rng, prefix, [cap] * B, page)
    cache = filled(fa, rng, fmt, n_pages, Hkv, page, d)
    inv, axis = fa.rotary_frequencies(d // 2, [d // 8, 3 * d // 16, 3 * d // 16])
    pt, pl, t = ints([int(x) for x in shared]), ints([prefix]), ints(table.tolist())
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    weight = torch.zeros(B, Hkv, table.shape[1] * page, device=DEV)
    cu = ints([Nq * i for i in range(B + 1)])
    held = 0
    evictions = 0
    for step in range(2 * steps):
        qkv = torch.from_numpy(rng.standard_normal((B * Nq, H + 2 * Hkv, d))).to(DT[dtype]).to(DEV)
        pos = ints(rng.integers(0, 40, (3, B * Nq)).tolist()) + prefix + Nq * step
        q, k = fa.rotary(qkv[:, :H], qkv[:, H : H + Hkv], pos, inv, axis)
        check_rotary(q, qkv[:, :H], pos, inv, axis, False, False)
        before = as_ref(cache)
        fa.kvq8_append(cache, k, qkv[:, H + Hkv :], t, cu, lens, Nq)
        ref.append(before[0], before[1], fmt, k.cpu().double().numpy(), table, cu.tolist(), lens.tolist())
        ref.append(before[2], before[3], fmt, qkv[:, H + Hkv :].cpu().double().numpy(), table, cu.tolist(), lens.tolist())
        check_cache(cache, before)
        lens = lens + Nq
        held += Nq
        rows = q.view(B, Nq, H, d).transpose(1, 2).contiguous()
        out, lse = fa.attention_kvq8_prefix(rows, cache, pt, pl, t, lens, causal=Nq > 1, max_prefix=prefix)
        check(rows, cache, shared, prefix, table, [held] * B, out, lse, 1 / math.sqrt(d), Nq > 1)
        was = weight.cpu().double().numpy()
        fa.kvq8_weights(rows, cache, t, lens, lse, weight, causal=Nq > 1)
        now = weight.cpu().double().numpy()
        kc, ks, _, _ = as_ref(cache)
        for s in (0, B - 1):
            add, bound = er.weights(rows[s].cpu().double().numpy(), ref.gather(kc, ks, table[s], held),
                                    lse[s].cpu().double().numpy(), d ** -0.5, Nq > 1)
            assert np.all(np.abs(now[s, :, :held] - was[s, :, :held] - add) <= bound + 2.0 ** -23 * now[s, :, :held])
        if held > budget + over - Nq:
            want, w = as_ref(cache), weight.cpu().numpy()
            lens, kept, weight = fa.kvq8_evict(cache, t, lens, weight, budget, 7)
            at = [[er.keep_positions(w[s, h, :held], budget, 7) for h in range(Hkv)] for s in range(B)]
            assert kept.tolist() == at and lens.tolist() == [budget] * B
            er.evict(want[0], want[1], fmt, table, [held] * B, at)
            er.evict(want[2], want[3], fmt, table, [held] * B, at)
            check_cache(cache, want)
            held = budget
            evictions += 1
    assert evictions > 0
    status_ok(fa)


def test_calls_at_once(fa):
    """Each operator on a stream of its own, over the same cache, gives what it gives alone."""
    rng = np.random.default_rng(3)
    prefix, lens, page, d = 3000, [400, 33, 700, 5, 0, 64, 911, 100], 16, 128
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, "int8", n_pages, 4, page, d)
    other = fa.KVCacheQ8(*(x.clone() for x in cache))
    q = torch.randn(8, 16, 1, d, device=DEV).bfloat16()
    q2 = torch.randn(8, 16, 1, d, device=DEV).bfloat16()
    pt, pl, t, n = ints([int(x) for x in shared]), ints([prefix]), ints(table.tolist()), ints(lens)
    w = torch.from_numpy(make_weights(rng, 8, 4, table.shape[1] * page, "spread")).to(DEV)
    plan = fa.fa_kvq8_prefix_plan(8, 16, 4, 1, prefix, max(lens), d)
    kw = dict(max_prefix=prefix, max_len=max(lens), n_splits=max(plan[0], 4), n_parts=plan[1])

    def calls(streams):
        got, acc = [None] * 4, w.clone()
        mine = fa.KVCacheQ8(*(x.clone() for x in other))
        for s in set(streams):
            s.wait_stream(torch.cuda.current_stream())
        got[0] = fa.attention_kvq8_prefix(q, cache, pt, pl, t, n, stream=streams[0], **kw)
        got[1] = fa.attention_kvq8_prefix(q2, cache, pt, pl, t, n, stream=streams[1], **kw)
        fa.kvq8_weights(q, cache, t, n, lse0, acc, stream=streams[2])
        got[2] = (acc,)
        got[3] = (*fa.kvq8_evict(mine, t, n, w, 64, 10, stream=streams[3]), *mine)
        for s in set(streams):
            s.synchronize()
        return [x for g in got for x in g]

    lse0 = fa.attention_kvq8(q, cache, t, n)[1]
    one = torch.cuda.Stream()
    want = calls([one] * 4)
    for _ in range(5):
        for x, y in zip(want, calls([torch.cuda.Stream() for _ in range(4)])):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    status_ok(fa)


def test_two_graphs_in_turn(fa):
    """Graphs captured apart have workspaces of their own: replayed in any order they give the same bits."""
    rng = np.random.default_rng(4)
    prefix, lens, page, d = 1500, [100, 260, 31], 32, 64
    shared, table, n_pages = tables(rng, prefix, lens, page)
    cache = filled(fa, rng, "e4m3", n_pages, 2, page, d)
    pt, pl, t, n = ints([int(x) for x in shared]), ints([prefix]), ints(table.tolist()), ints(lens)
    graphs, outs, want = [], [], []
    for splits, parts in ((3, 2), (5, 0)):
        q = torch.randn(3, 20, 2, d, device=DEV).half()
        kw = dict(causal=True, max_prefix=prefix, max_len=260, n_splits=splits, n_parts=parts)
        want.append(fa.attention_kvq8_prefix(q, cache, pt, pl, t, n, **kw)[0])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.attention_kvq8_prefix(q, cache, pt, pl, t, n, **kw)[0])
        graphs.append(g)
        outs.append(q)  # stays alive
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        outs[0].zero_()
        outs[2].zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[2], want[1])
    status_ok(fa)


def test_offsets_past_32_bits(fa):
    """A cache of more than 4 GB of codes whose last pages are the ones in use."""
    page, Hkv, d, H = 128, 8, 128, 16
    n_pages = 2 ** 32 // (page * Hkv * d) + 40
    rng = np.random.default_rng(5)
    prefix, lens = 900, [300, 129]
    shared, table, used = tables(rng, prefix, lens, page, spare=0)
    small = filled(fa, rng, "int8", used, Hkv, page, d)
    big = fa.kv_cache_q8(n_pages, Hkv, page, d, CODE["int8"], DEV)
    at = n_pages - used
    for x, y in zip(big, small):
        x[at:] = y
    q = torch.from_numpy(rng.standard_normal((2, H, 1, d))).bfloat16().to(DEV)
    far = np.where(table < used, table + at, table)
    pt, pl, n = ints([int(x) + at for x in shared]), ints([prefix]), ints(lens)
    for splits in ((0, 1), (3, 0)):
        out, lse = fa.attention_kvq8_prefix(q, big, pt, pl, ints(far.tolist()), n, n_splits=splits[0], n_parts=splits[1])
        check(q, small, shared, prefix, table, lens, out, lse, d ** -0.5, False)
    w = torch.from_numpy(make_weights(rng, 2, Hkv, table.shape[1] * page, "spread")).to(DEV)
    _, lse = fa.attention_kvq8(q, small, ints(table.tolist()), n)
    a, b = w.clone(), w.clone()
    fa.kvq8_weights(q, small, ints(table.tolist()), n, lse, a)
    fa.kvq8_weights(q, big, ints(far.tolist()), n, lse, b)
    assert torch.equal(a, b)
    one = fa.kvq8_evict(small, ints(table.tolist()), n, w, 150, 20)
    two = fa.kvq8_evict(big, ints(far.tolist()), n, w, 150, 20)
    for x, y in zip(one, two):
        assert torch.equal(x, y)
    for x, y in zip(big, small):
        assert torch.equal(x[at:].view(torch.uint8), y.view(torch.uint8))
    assert int(big.k_codes[: at].view(torch.int64).count_nonzero()) == 0
    status_ok(fa)


def test_weights_and_eviction_ignore_what_lies_behind(fa):
    """Slots behind the lengths hold NaN codes, pages of nobody too; many sequences, most of them short or empty."""
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 40, 100)] + [300, 0, 257]
    page, d, Hkv = 16, 64, 2
    table, n_pages = random_table(rng, [max(n, 1) for n in lens], page)
    cache = filled(fa, rng, "e4m3", n_pages, Hkv, page, d)
    used = torch.zeros(n_pages, page, dtype=torch.bool, device=DEV)
    for s, n in enumerate(lens):
        for i in range(n):
            used[int(table[s][i // page]), i % page] = True
    for codes in (cache.k_codes, cache.v_codes):
        codes.view(torch.uint8)[(~used)[:, None].expand(n_pages, Hkv, page)] = 0x7F
    q = torch.randn(len(lens), 4, 1, d, device=DEV).half()
    t, n = ints(table.tolist()), ints(lens)
    _, lse = fa.attention_kvq8(q, cache, t, n)
    weight = torch.zeros(len(lens), Hkv, table.shape[1] * page, device=DEV)
    fa.kvq8_weights(q, cache, t, n, lse, weight)
    assert torch.isfinite(weight).all()
    total = weight.sum(-1).cpu()
    assert torch.allclose(total, torch.tensor([[2.0 * (m > 0)] * Hkv for m in lens]), rtol=1e-3)
    w = weight.cpu().numpy()
    raw = [x.clone() for x in (cache.k_codes.view(torch.uint8), cache.v_codes.view(torch.uint8))]
    new, kept, _ = fa.kvq8_evict(cache, t, n, weight, 20, 5)
    assert new.tolist() == [min(m, 20) for m in lens]
    for s, m in enumerate(lens):
        for h in range(Hkv):
            at = er.keep_positions(w[s, h, :m], 20, 5)
            assert kept[s, h, : len(at)].tolist() == at
        for i in range(20, table.shape[1] * page):  # slots that take nothing are as they were
            p = int(table[s][i // page])
            if p < n_pages:
                assert torch.equal(cache.k_codes.view(torch.uint8)[p, :, i % page], raw[0][p, :, i % page])
    status_ok(fa)


def test_budget_beyond_the_tables_reach(fa):
    rng = np.random.default_rng(7)
    table, n_pages = random_table(rng, [30, 16], 16)
    cache = filled(fa, rng, "int8", n_pages, 1, 16, 64)
    want = as_ref(cache)
    w = torch.rand(2, 1, 32, device=DEV)
    new, kept, out = fa.kvq8_evict(cache, ints(table.tolist()), ints([30, 16]), w, 100, 100)
    assert new.tolist() == [30, 16] and kept[0, 0].tolist() == list(range(30)) + [-1] * 70
    assert torch.equal(out[0, 0, :30], w[0, 0, :30]) and (out[0, 0, 30:] == 0).all()
    check_cache(cache, want)
    status_ok(fa)
