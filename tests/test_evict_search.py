"""The selection's search takes exactly the positions that the definition names, whatever the weights are. CPU only."""
import numpy as np
import pytest

import evict_ref as er
import evict_search as es

KINDS = ["positive", "nan", "nan_low", "nan_zero", "nan_inf", "few_nan", "all_nan", "ties", "odd", "one"]


def weights(rng, n, kind):
    w = np.exp(rng.standard_normal(n) * 3).astype(np.float32)
    if kind.startswith("nan"):
        w[rng.random(n) < 0.5] = np.nan
        extra = {"nan": None, "nan_low": np.float32(1e-42), "nan_zero": 0.0, "nan_inf": -np.inf}[kind]
        if extra is not None:
            w[rng.integers(0, n)] = extra
    elif kind == "few_nan":
        w[rng.random(n) < 0.05] = np.nan
    elif kind == "all_nan":
        w[:] = np.nan
    elif kind == "ties":
        w = rng.integers(0, 3, n).astype(np.float32) - 1
    elif kind == "odd":
        for x in (-0.0, 0.0, np.nan, np.inf, -np.inf, -3.5, 1e-42, np.float32(3e38)):
            w[rng.random(n) < 0.08] = x
    elif kind == "one":
        w[:] = 0.25
        w[rng.integers(0, n)] = 0.5
    return w


@pytest.mark.parametrize("kind", KINDS)
def test_search_takes_what_the_definition_names(kind):
    rng = np.random.default_rng(KINDS.index(kind))
    for n in (2, 3, 17, 150, 1000, 2500):
        w = weights(rng, n, kind)
        for need in sorted({1, 2, n // 10, n // 3, n // 2, n - 1} & set(range(1, n))):
            assert es.select(w, need) == er.keep_positions(w, need, 0), (n, need)


def test_a_bin_end_that_wraps_is_found():
    """More NaN than places beside weights above 0: with the end of the top bin formed in 32 bits every NaN is taken."""
    w = np.full(1050, np.nan, np.float32)
    w[950:] = np.exp(np.random.default_rng(0).standard_normal(100))
    assert len(es.select(w, 900, es.bin_end_wrapped)) > 900
    assert es.select(w, 900) == list(range(900))
    w = np.exp(np.random.default_rng(1).standard_normal(1000)).astype(np.float32)
    w[::2] = np.nan
    assert len(es.select(w, 100, es.bin_end_wrapped)) == 500
    assert es.select(w, 100) == list(range(0, 200, 2))
