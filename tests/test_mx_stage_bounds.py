"""What the FFN's stage-by-stage check can see at large sizes: faults planted
in the oracle lie far outside its tolerances (no GPU needed)."""
import numpy as np
import pytest

from oracle import mx_oracle as M

D, F, ROWS = 2432, 1536, 8


@pytest.fixture(scope="module")
def case():
    rng = np.random.default_rng(0)
    x = M.exact_rows(rng, ROWS, D)
    wg, wu = (M.exact_rows(rng, F, D, -8) for _ in range(2))
    wd = M.rounded(rng.standard_normal((D, F)) * 0.05)
    q, lo, hi = M.hidden(x, wg, wu)
    y, tol = M.product(q, wd)
    return x, wg, wu, wd, q, lo, hi, y, tol + M.half_step(np.abs(y) + tol, 2.0 ** -10, 2.0 ** -24)


def test_inputs_are_their_own_form_and_their_sums_exact(case):
    x, wg, wu = case[:3]
    for v in (x, wg, wu):
        np.testing.assert_array_equal(M.rounded(v), v)
        assert len(np.unique(M.scale_bytes(v))) == 1
    unit = 2.0 ** -10                                        # 1/4 of the two scales' product
    for w in (wg, wu):
        assert ((np.abs(x) @ np.abs(w).T) / unit < 2.0 ** 24).all() and ((x @ w.T) / unit == np.round((x @ w.T) / unit)).all()


def test_tolerances_are_small(case):
    q, lo, hi, y, lim = case[4:]
    assert (lo != hi).mean() < 1e-3
    assert np.median(lim) < 0.01 * np.median(np.abs(y))


def test_planted_faults_are_seen(case):
    x, wg, wu, wd, q, lo, hi, y, lim = case
    short = M.hidden(x[:, :-32], wg[:, :-32], wu[:, :-32])[0]          # the last 32 of d left out
    assert ((short < lo) | (short > hi)).mean() > 0.1
    g = x @ wg.T
    h = g / (1 + np.exp(-g)) * (x @ wu.T)
    assert ((h < lo) | (h > hi)).mean() > 0.5                          # h not quantised
    swapped = M.hidden(x, wu, wg)[0]                                   # gate and up exchanged
    assert ((swapped < lo) | (swapped > hi)).mean() > 0.5
    assert (np.abs(q[:, :-32] @ wd[:, :-32].T - y) > lim).mean() > 0.5   # the last 32 of F left out
    assert (np.abs(h @ wd.T - y) > lim).mean() > 0.5                   # the down product of h itself
