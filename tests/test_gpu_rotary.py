"""GPU parity of the rotary positions against the definition in 64 bits (angles in extended precision).

Tolerance, per value, from the arithmetic. y = x1 c -+ x2 s with c, s within 2^-22 of exact (sincospi's two units, the
fp32 rounding of an angle of at most half a turn, pi 2^-25), or further at far positions by the angle's own error,
|p f| 2^-53 radians from the 53 bits of f / 2 pi; two fp32 roundings of at most 2^-24 (|x1| + |x2|) each; one rounding
to the output's type, half a step of it relative, or half of the smallest subnormal number. So
    |y - ref| <= (|x1| + |x2|) (2^-21 + |p f| 2^-53) + half_step |ref| + 2^-25 for fp16, 2^-134 for bf16.
"""
import numpy as np
import pytest
import torch

import evict_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


def check(got, x, pos, inv, axis, inverse, heads_first):
    """x, got: torch tensors [total, H, d], or [B, H, N, d]."""
    a, g = x.detach().cpu().double().numpy(), got.detach().cpu().double().numpy()
    p = pos.cpu().numpy()
    if heads_first:
        a, g = a.transpose(0, 2, 1, 3), g.transpose(0, 2, 1, 3)
    inv, axis = inv.numpy(), axis.numpy()
    want = ref.rotary(a, p, inv, axis, inverse)
    r = len(inv)
    if r * 2 < a.shape[-1]:
        assert np.array_equal(g[..., 2 * r :], a[..., 2 * r :])
    far = np.zeros(p.shape[1:] + (1, r))
    for i in range(r):
        far[..., 0, i] = np.abs(p[axis[i]].astype(np.float64) * inv[i]) * 2.0 ** -53
    mag = (np.abs(a[..., :r]) + np.abs(a[..., r : 2 * r])) * (2.0 ** -21 + far)
    half = torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == torch.float16 else 2.0 ** -134
    tol = np.concatenate([mag, mag], -1) + half * np.abs(want[..., : 2 * r]) + tiny
    assert np.all(np.abs(g[..., : 2 * r] - want[..., : 2 * r]) <= tol)


def positions(rng, axes, *tokens, far=5000):
    return torch.from_numpy(rng.integers(0, far, (axes, *tokens))).int().to(DEV)


CASES = [  # total, Hq, Hk, d, pairs, sections
    (1, 1, 1, 64, 32, [8, 12, 12]), (1, 8, 2, 128, 64, [16, 24, 24]), (7, 5, 1, 128, 24, [24]), (33, 3, 3, 64, 8, [3, 0, 5]),
    (129, 32, 8, 128, 64, [16, 24, 24]), (257, 7, 0, 64, 16, [4, 4, 4, 4]), (1000, 4, 1, 128, 40, [10, 15, 15]),
]


@pytest.mark.parametrize("total,Hq,Hk,d,pairs,sections", CASES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inverse", [False, True])
def test_packed_matches_the_definition(fa, total, Hq, Hk, d, pairs, sections, dtype, inverse):
    rng = np.random.default_rng(total + d)
    wide = torch.from_numpy(rng.standard_normal((total, Hq + 2 * Hk + 1, d + 8))).to(DT[dtype]).to(DEV)
    q, k = wide[:, :Hq, 8:], wide[:, Hq : Hq + Hk, :d] if Hk else None
    inv, axis = fa.rotary_frequencies(pairs, sections, theta=1e6 if inverse else 1e4, interleaved=inverse)
    pos = positions(rng, len(sections), total, far=100000)
    turn = fa.rotary_backward if inverse else fa.rotary
    before = wide.clone()
    gq, gk = turn(q, k, pos, inv, axis)
    assert torch.equal(wide, before) and gq.is_contiguous() and (gk is None) == (Hk == 0)
    check(gq, q, pos, inv, axis, inverse, False)
    if Hk:
        check(gk, k, pos, inv, axis, inverse, False)
    iq, ik = turn(q, k, pos, inv, axis, inplace=True)  # the same numbers, in the wider buffer, and nothing else in it
    assert iq is q and ik is k and torch.equal(q, gq) and (Hk == 0 or torch.equal(k, gk))
    after = wide.clone()
    after[:, :Hq, 8:] = before[:, :Hq, 8:]
    if Hk:
        after[:, Hq : Hq + Hk, :d] = before[:, Hq : Hq + Hk, :d]
    assert torch.equal(after, before)


@pytest.mark.parametrize("B,Hq,Hk,N,d", [(1, 1, 1, 1, 64), (3, 4, 2, 17, 128), (2, 16, 16, 300, 64), (5, 6, 1, 9, 128)])
@pytest.mark.parametrize("transposed", [False, True])
def test_heads_first_matches_the_definition(fa, B, Hq, Hk, N, d, transposed):
    rng = np.random.default_rng(B + N)
    inv, axis = fa.rotary_frequencies(d // 2, [d // 8, 3 * d // 16, 3 * d // 16], interleaved=True)
    pos = positions(rng, 3, B, N)

    def tensor(h):
        shape = (B, N, h, d) if transposed else (B, h, N, d)
        t = torch.from_numpy(rng.standard_normal(shape)).to(torch.bfloat16).to(DEV)
        return t.transpose(1, 2) if transposed else t

    q, k = tensor(Hq), tensor(Hk)
    gq, gk = fa.rotary(q, k, pos, inv, axis)
    check(gq, q, pos, inv, axis, False, True)
    check(gk, k, pos, inv, axis, False, True)


def test_keys_that_all_heads_share(fa):
    """Input rows repeated by a stride of zero are read as they are; they cannot be turned in place."""
    rng = np.random.default_rng(0)
    k = torch.from_numpy(rng.standard_normal((6, 1, 64))).half().to(DEV).expand(6, 4, 64)
    q = torch.from_numpy(rng.standard_normal((6, 4, 64))).half().to(DEV)
    inv, axis = fa.rotary_frequencies(32)
    pos = positions(rng, 1, 6)
    _, gk = fa.rotary(q, k, pos, inv, axis)
    check(gk, k, pos, inv, axis, False, False)
    with pytest.raises(ValueError):
        fa.rotary(q, k, pos, inv, axis, inplace=True)


@pytest.mark.parametrize("place", [0, 1, -1, 2 ** 20 + 1, -(2 ** 24) - 3, 2 ** 31 - 1, -(2 ** 31)])
def test_far_positions(fa, place):
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.standard_normal((3, 2, 128))).bfloat16().to(DEV)
    inv, axis = fa.rotary_frequencies(64, [32, 32])
    inv[5] = -inv[5]
    inv[6] = 0.0
    inv[7] = 6.5  # more than a turn
    pos = torch.tensor([[place, place, 0], [0, place, place]], dtype=torch.int32, device=DEV)
    got, _ = fa.rotary(q, None, pos, inv, axis)
    check(got, q, pos, inv, axis, False, False)
    if place == 0:
        assert torch.equal(got, q)


def test_special_values(fa):
    """NaN and infinities stay in their pair; a pair with position 0 is left as it is; fp16's largest numbers."""
    q = torch.randn(4, 1, 64, device=DEV).half()
    q[0, 0, 3], q[1, 0, 40], q[2, 0, 5] = float("nan"), float("inf"), 65504.0
    inv, axis = fa.rotary_frequencies(32)
    got, _ = fa.rotary(q, None, positions(np.random.default_rng(0), 1, 4, far=50) + 1, inv, axis)
    bad = ~torch.isfinite(got)
    for row, i in ((0, 3), (1, 8)):
        assert bad[row, 0, [i, i + 32]].all()
        bad[row, 0, [i, i + 32]] = False
    bad[2, 0, [5, 37]] = False  # 65504 sin may round to either side
    assert not bad.any()


def test_gradient_against_differences(fa):
    """sum(g . rotary(x)) is linear in x: its difference along any direction v is sum(rotary_backward(g) . v)."""
    rng = np.random.default_rng(9)
    inv, axis = fa.rotary_frequencies(64, [16, 24, 24])
    pos = positions(rng, 3, 2, 50)
    x, v, g = (torch.from_numpy(rng.standard_normal((2, 3, 50, 128))).half().to(DEV) for _ in range(3))
    dx, _ = fa.rotary_backward(g, None, pos, inv, axis)
    plus, minus = x.clone(), x.clone()
    idx = torch.from_numpy(rng.integers(0, 128, (20,))).to(DEV)
    for i in idx.tolist():  # one element of each row at a time
        plus.copy_(x)
        minus.copy_(x)
        plus[..., i] += 1.0
        minus[..., i] -= 1.0
        step = (plus[..., i].double() - minus[..., i].double())
        up, down = (fa.rotary(t, None, pos, inv, axis)[0].double() for t in (plus, minus))
        slope = ((up - down) * g.double()).sum(-1)
        # two outputs a row depend on the element, each off by half a step of its size (at most 2^-11 (|x| + 1) sqrt 2)
        j = (i + 64) % 128
        tol = 2 * 2.0 ** -11 * (plus[..., [i, j]].abs().sum(-1) + minus[..., [i, j]].abs().sum(-1)).double() * g[..., [i, j]].abs().sum(-1).double()
        tol = tol + 2.0 ** -10 * (g[..., i].abs() + g[..., j].abs()).double() * step
        assert torch.all((slope - dx[..., i].double() * step).abs() <= tol)


def test_stream_graph_and_larger_launch(fa):
    rng = np.random.default_rng(4)
    inv, axis = fa.rotary_frequencies(64, [16, 24, 24])
    pos = positions(rng, 3, 5000)
    qkv = torch.randn(5000, 12, 128, device=DEV).bfloat16()
    q, k = qkv[:, :8], qkv[:, 8:10]
    want = fa.rotary(q, k, pos, inv, axis)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.rotary(q, k, pos, inv, axis, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.rotary(q, k, pos, inv, axis)
    inv.zero_()  # the frequencies were read during the call
    pos.copy_(pos + 7)
    graph.replay()
    torch.cuda.synchronize()
    inv, _ = fa.rotary_frequencies(64, [16, 24, 24])
    again = fa.rotary(q, k, pos, inv, axis)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    assert fa.fa_get_device_status() == fa.FA_OK
