"""Rotary positions refuse outputs that lie on another tensor, on the host before anything is launched; and the test of
rows against rows, compiled by itself, gives what their bytes say. CPU only."""
import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "io_aware_exact_13_gb300", "csrc")


@pytest.fixture(scope="module")
def fa():
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    return mod


def rotary(fa, q, q_out, k, k_out, q_strides, k_strides, N=3, Hq=2, Hk=2, d=64, B=1, positions=0x40000000, name="fa_rotary"):
    six = lambda s: (ctypes.c_longlong * 6)(*s, *s) if len(s) == 3 else (ctypes.c_longlong * 6)(*s)
    f, a = (ctypes.c_double * 64)(*[0.5] * 64), (ctypes.c_int * 64)(*[0] * 64)
    p = [ctypes.c_void_p(x) for x in (q, q_out, k, k_out, positions)]
    return getattr(fa.lib, name)(p[0], p[1], six(q_strides), Hq, p[2], p[3], six(k_strides), Hk, p[4], 1, f, a, 32, B, N, d, 0, None)


@pytest.mark.parametrize("name", ["fa_rotary", "fa_rotary_fp16"])
def test_outputs_on_other_tensors_are_refused(fa, name):
    A, B_, C, D = 0x1000000, 0x2000000, 0x3000000, 0x3800000
    s, size = (0, 128, 64), 3 * 128 * 2  # packed [3][2][64], its bytes
    for off in (16, 128, 256, size - 16, -16, -128, 16 - size):
        assert rotary(fa, A, C + off, C, D, s, s, name=name) == fa.FA_ERR_ARG  # q_out within k
        assert rotary(fa, A, C, B_, A + off, s, s, name=name) == fa.FA_ERR_ARG  # k_out within q
        assert rotary(fa, A, C, B_, C + off, s, s, name=name) == fa.FA_ERR_ARG  # the outputs on each other
        assert rotary(fa, A, A + off, B_, D, s, s, name=name) == fa.FA_ERR_ARG  # q_out behind its own input
        assert rotary(fa, A, C, B_, B_ + off, s, s, name=name) == fa.FA_ERR_ARG
    for at in (A, B_):
        assert rotary(fa, A, A, B_, B_, s, s, positions=at, name=name) == fa.FA_ERR_ARG  # on the positions
        assert rotary(fa, A, A, B_, B_, s, s, positions=at + size - 4, name=name) == fa.FA_ERR_ARG
    assert rotary(fa, A, A, A + 128, A + 128, (0, 512, 64), (0, 512, 64), name=name) == fa.FA_ERR_ARG  # heads of one buffer: 0, 1 and 1, 2
    assert rotary(fa, A, A, A + 64, A + 64, (0, 512, 128), (0, 512, 128), name=name) == fa.FA_ERR_ARG  # half a row apart
    assert rotary(fa, A, C, C + 8192, D, s, (0, -4096, 64, 0, 128, 64), name=name) == fa.FA_ERR_ARG  # an input that runs backwards


@pytest.mark.parametrize("name", ["fa_rotary", "fa_rotary_fp16"])
def test_strides_out_of_proportion_are_refused(fa, name):
    A, B_ = 0x1000000, 0x2000000
    for s in ((0, 1 << 41, 64), (0, -(1 << 41), 64), (0, 128, 1 << 60), (0, -(2 ** 63), 64)):
        assert rotary(fa, A, B_, A, B_, (*s, 0, 128, 64), (*s, 0, 128, 64), name=name) == fa.FA_ERR_SHAPE
    # with many entries even smaller ones
    assert rotary(fa, A, B_, A, B_, (0, 1 << 39, 64, 0, 1 << 39, 64), (0, 128, 64), N=1 << 20, name=name) == fa.FA_ERR_SHAPE


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    at = tmp_path_factory.mktemp("rows")
    src = at / "rows.cpp"
    src.write_text('''#include "rows.h"
extern "C" int meet(long long a, long long ra, const long long *sa, const long long *ca, long long b, long long rb,
                    const long long *sb, const long long *cb) {
    fa::Rows x((void *)a, ra), y((void *)b, rb);
    for (int i = 0; i < 3; ++i)
        if (!x.add(sa[i], ca[i]) || !y.add(sb[i], cb[i])) return -1;
    return fa::rows_meet(x, y);
}''')
    lib = at / "rows.so"
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).meet
    three = lambda v: (ctypes.c_longlong * 3)(*v)

    def call(a, b):  # each (first, row, strides, counts)
        return f(*(ctypes.c_longlong(x) if np.isscalar(x) else three(x) for x in (*a, *b)))

    return call


def bytes_of(first, row, strides, counts):
    return {first + sum(i * s for i, s in zip(at, strides)) + j for at in itertools.product(*(range(c) for c in counts)) for j in range(row)}


def test_rows_meet_where_their_bytes_do(meet):
    """Random strides of either sign, zeros, nested or not, alike in both or not, of two rows lengths."""
    rng = np.random.default_rng(0)
    met = 0
    for _ in range(6000):
        row = int(rng.choice([4, 8]))
        both = [int(x) for x in rng.choice([0, 4, 8, 12, 16, 24, 40, 64, 100, -8, -16, -40], 3)]
        a, b = [], []
        for t in (a, b):
            strides = both if rng.random() < 0.5 else [int(x) for x in rng.choice([0, 4, 8, 16, 20, 48, 96, 160, -12, -64], 3)]
            t += [1000 + int(rng.integers(-60, 60)) * 4, row, strides, [int(x) for x in rng.integers(1, 5, 3)]]
        want = bool(bytes_of(*a) & bytes_of(*b))
        met += want
        assert meet(a, b) == want, (a, b)
        assert meet(b, a) == want, (a, b)
    assert 1000 < met < 5000


def test_layouts_in_use_do_not_meet(meet):
    N, H, G, d = 30011, 32, 8, 256  # d: bytes of a row
    W = (H + 2 * G) * d
    q = (1 << 30, d, (W, d, 0), (N, H, 1))
    assert meet(q, ((1 << 30) + H * d, d, (W, d, 0), (N, G, 1))) == 0  # one packed buffer
    assert meet(q, ((1 << 30) + (H - 1) * d, d, (W, d, 0), (N, G, 1))) == 1
    assert meet((1 << 30, d, (W, 2 * d, 0), (N, G, 1)), ((1 << 30) + d, d, (W, 2 * d, 0), (N, G, 1))) == 0  # heads in turn
    n = N * d  # heads first
    assert meet((1 << 30, d, (W * N, n, d), (4, H, N)), ((1 << 30) + H * n, d, (W * N, n, d), (4, G, N))) == 0
    assert meet((1 << 30, d, (W * N, n, d), (4, H, N)), ((1 << 30) + H * n, d, (W * N, d, 0), (4, N, 1))) == 0  # a single head
    assert meet(q, ((1 << 40), d, (W, d, 0), (N, G, 1))) == 0


def test_what_cannot_be_told_in_time_counts_as_overlap(meet):
    """Rows of one tensor between every second of the other's, at more than 4096 places to look at."""
    for count, want in ((3000, 0), (5000, 1)):
        assert meet((0, 16, (1000, 0, 0), (2 * count, 1, 1)), (500, 16, (2000, 0, 0), (count, 1, 1))) == want
