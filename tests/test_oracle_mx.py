"""Pins of the MXFP4 and scored-router oracle: hand values, layout positions,
brute force (no GPU needed)."""
import itertools

import numpy as np
import pytest

from oracle import mx_oracle as M


def test_grid_values_are_kept_and_midpoints_go_to_the_even_code():
    v = np.zeros(32)
    v[:8] = M.GRID                                # largest magnitude 6: scale 2^0
    code, byte = M.quantize(v[None])
    assert byte[0, 0] == 127
    assert code[0, :8].tolist() == list(range(8))
    v[8:15] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    code, _ = M.quantize(v[None])
    assert code[0, 8:15].tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert M.values(code, byte)[0, 8:15].tolist() == [0, 1, 1, 2, 2, 4, 4]


@pytest.mark.parametrize("amax,byte", [(1.0, 125), (1.999, 125), (2.0, 126), (7.9, 127), (8.0, 128), (0.0, 0),
                                       (2.0 ** -140, 0), (3e38, 252), (np.inf, 255), (np.nan, 255)])
def test_scale_byte(amax, byte):
    v = np.zeros((1, 32))
    v[0, 5] = -amax
    assert M.scale_bytes(v)[0, 0] == byte


def test_saturation_and_sign():
    v = np.zeros((1, 32))
    v[0, 0], v[0, 1], v[0, 2] = 7.99, -7.99, -0.3   # 7.99 has scale 2^0 and saturates at 6
    code, byte = M.quantize(v)
    assert M.values(code, byte)[0, :3].tolist() == [6, -6, -0.5]


def test_rounding_is_nearest_by_brute_force():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((40, 32)) * np.exp2(rng.integers(-20, 20, (40, 1)))
    q = M.rounded(v)
    unit = np.exp2(M.scale_bytes(v).astype(float) - 127)
    grid = np.concatenate([-M.GRID[::-1], M.GRID])
    best = np.min(np.abs(v[:, :, None] - grid * unit[:, :, None]), axis=-1)
    np.testing.assert_array_equal(np.abs(v - q), best)


def test_layout_positions():
    assert M.pack_codes(np.array([[1, 2, 15, 0]], dtype=np.uint8)).tolist() == [[0x21, 0x0F]]
    assert M.scale_at(0, 0, 256) == 0
    assert M.scale_at(0, 3, 256) == 3
    assert M.scale_at(33, 1, 256) == 16 + 4 + 1
    assert M.scale_at(5, 4, 256) == 512 + 5 * 16
    assert M.scale_at(128, 0, 256) == 2 * 512
    g, u = M.gate_up_rows(64)
    assert (g[0], u[0], g[31], u[31], g[32], u[32]) == (0, 32, 31, 63, 64, 96)
    w = np.random.default_rng(1).standard_normal((256, 256))
    raw = M.matrix(w)
    code, byte = M.quantize(w)
    np.testing.assert_array_equal(M.unpack_codes(raw[:256 * 128].reshape(256, 128)), code)
    where = {M.scale_at(r, b, 256) for r in range(256) for b in range(8)}
    assert where == set(range(256 * 8))


@pytest.mark.parametrize("scoring,groups,kept,top", [("softmax", 1, 1, 1), ("sigmoid", 4, 2, 1), ("sigmoid", 3, 2, 2),
                                                      ("softmax", 4, 3, 2)])
def test_route_scored_brute_force(scoring, groups, kept, top):
    rng = np.random.default_rng(2)
    T, d, E, k = 9, 32, 12, 3
    x, w = rng.standard_normal((T, d)), rng.standard_normal((E, d)) * 0.2
    bias = rng.standard_normal(E) * 0.1
    idx, wt, s = M.route_scored(x, w, k, scoring, bias, groups, kept, top, True, 2.5)
    l = x @ w.T
    want = 1 / (1 + np.exp(-l)) if scoring == "sigmoid" else np.exp(l) / np.exp(l).sum(1, keepdims=True)
    np.testing.assert_allclose(s, want, rtol=1e-12)
    np.testing.assert_allclose(wt.sum(1), 2.5)
    c = want + bias
    gs = E // groups
    for t in range(T):
        # the best set of groups, then the best ordered k of their experts, over all of them
        by = [np.sort(c[t, g * gs:(g + 1) * gs])[-top:].sum() for g in range(groups)]
        best = max(itertools.combinations(range(groups), kept), key=lambda q: sum(by[g] for g in q))
        ok = [e for g in best for e in range(g * gs, (g + 1) * gs)]
        picks = max(itertools.combinations(ok, k), key=lambda q: sum(c[t, e] for e in q))
        assert sorted(picks) == sorted(idx[t])
        assert (np.diff(c[t, idx[t]]) <= 0).all()


def test_route_scored_ties_and_masks():
    x = np.ones((1, 32))
    w = np.zeros((8, 32))
    idx, wt, _ = M.route_scored(x, w, 3, "sigmoid")
    assert idx.tolist() == [[0, 1, 2]] and np.allclose(wt, 1 / 3)
    bias = np.full(8, -np.inf)
    bias[[5, 7]] = 0
    idx, _, _ = M.route_scored(x, w, 3, "sigmoid", bias)
    assert idx.tolist() == [[5, 7, 0]]
    # four groups of two, equal sums: the lower groups stay
    idx, _, _ = M.route_scored(x, w, 3, "sigmoid", None, 4, 2, 2)
    assert idx.tolist() == [[0, 1, 2]]


def test_ffn_bound_covers_an_fp32_evaluation():
    rng = np.random.default_rng(3)
    x = M.rounded(rng.standard_normal((6, 128)))
    wg, wu, wd = (M.rounded(rng.standard_normal(s) * 0.05) for s in ((64, 128), (64, 128), (128, 64)))
    y, bound = M.ffn(x, wg, wu, wd)
    g = (x.astype(np.float32) @ wg.astype(np.float32).T).astype(np.float32)
    u = (x.astype(np.float32) @ wu.astype(np.float32).T).astype(np.float32)
    h = (g / (1 + np.exp(-g)) * u).astype(np.float64)
    got = M.rounded(h) @ wd.T
    assert (np.abs(got - y) <= bound).all()
    assert np.median(bound) < 1e-3 * np.median(np.abs(y))     # and says something
