"""The routers where squares, scores or sums leave fp32's range, against the
fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import mx_oracle as M
from quantized_moe_expert_histogram_b200 import build, moeq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moeq.load()


def swapped_ties(T, d, E, families, seed):
    """x in steps of 2^-4 and w in steps of 2^-26, so that every fp64 sum is
    exact in any order while the fp32 sums round; x is the same at 2i and
    2i + 1, and the rows of a family differ in which of these they swap
    (equal logits), every fourth of them also by a step in a few places (nearly
    equal ones)."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, d // 2, generator=g) * 16).round().clamp(-128, 128) / 16
    x = x.repeat_interleave(2, 1)
    base = (torch.randn(families, d // 2, 2, generator=g) * 0.02 * 2 ** 26).round()
    w = base[torch.arange(E) % families]
    swap = torch.rand(E, d // 2, generator=g) < 0.5
    w = torch.where(swap[..., None], w.flip(-1), w)
    w[torch.arange(E) // families % 4 == 3, ::61, 0] += 1
    return x, (w / 2 ** 26).reshape(E, d)


MAGNITUDES = [(0, 0), (-78, 70), (-78, 0), (-100, 98), (0, -80), (60, -84), (17, -83), (-76, -20)]


@pytest.mark.parametrize("T", [4, 60, 300])
@pytest.mark.parametrize("sx,sw", MAGNITUDES)
def test_near_ties_at_any_magnitude(sx, sw, T):
    """Activations of 2^sx and weights of 2^sw: their squares leave fp32's
    range below, the choice stays that of the fp64 logits."""
    x, w = swapped_ties(T, 1024, 64, 8, seed=50)
    x, w = (x * 2.0 ** sx).bfloat16(), w * 2.0 ** sw
    b = (torch.arange(64) % 8).float() / 1024
    for kw in (dict(), dict(scoring="sigmoid"), dict(scoring="sigmoid", n_groups=4, topk_groups=2),
               dict(scoring="sigmoid", bias=b)):
        idx, _ = moeq.moe_route_scored(x.cuda(), w.cuda(), 12, **{n: v.cuda() if n == "bias" else v for n, v in kw.items()})
        ref, _, _ = M.route_scored(x.double().numpy(), w.double().numpy(), 12,
                                   **{n: v.double().numpy() if n == "bias" else v for n, v in kw.items()})
        got = idx.cpu().numpy()
        if "bias" not in kw:
            np.testing.assert_array_equal(got, ref, err_msg=str(kw))
            continue
        # Choice values in fp64 are rounded themselves: exp errs by 2^-52 relative at most, 1 + exp, the division and
        # the bias addition by 2^-53 each, so a value in [0, 2) by less than 2^-52 (exp's error enters s as s (1 - s)
        # <= 1/4 of it), and two evaluations order values 2^-51 apart alike.  In steps of 2^-110 the logits of a family
        # differ by about 2^-50, their scores by a quarter of that: the oracle itself differs from an evaluation in 80
        # bits there.  So: the same picks but for values nearer than 2^-51.
        l = np.longdouble(x.double().numpy() @ w.double().numpy().T)
        c = 1 / (1 + np.exp(-l)) + np.longdouble(b.double().numpy())
        gap = np.abs(np.take_along_axis(c, got.astype(np.int64), 1) - np.take_along_axis(c, ref.astype(np.int64), 1))
        assert (gap <= 2.0 ** -51).all() and all(len(set(row)) == 12 for row in got.tolist())


@pytest.mark.parametrize("T", [4, 60, 300])
@pytest.mark.parametrize("sx,sw", MAGNITUDES)
def test_softmax_router_near_ties_at_any_magnitude(sx, sw, T):
    x, w = swapped_ties(T, 1024, 64, 8, seed=51)
    x, w = (x * 2.0 ** sx).bfloat16(), w * 2.0 ** sw
    idx, _ = moeq.moe_route_topk(x.cuda(), w.cuda(), None, 12)
    ref = O.topk_select(O.router_logits(x.double().numpy(), w.double().numpy()), 12)
    np.testing.assert_array_equal(idx.cpu().numpy(), ref)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("top", [-100.0, -500.0, -599.0, -601.0, -700.0, -709.5, -715.0, -730.0, -760.0])
def test_weights_of_scores_that_vanish(top, renorm, T):
    """Scores below fp32's and fp64's range, settled on fp32 logits: the
    weights are those of the fp64 scores, 0 where their sum is 0.  Logits are
    sums of two terms that every format here holds exactly; expf, the sum and
    the division round to less than 1e-6, and near e^-730 the scores themselves
    are multiples of 2^-1074, 5e-7 of them."""
    E, k = 32, 6
    x = torch.zeros(T, 64)
    x[:, 0], x[:, 1] = 1, torch.arange(T) % 3
    w = torch.zeros(E, 64)
    w[:, 0], w[:, 1] = top, -(torch.arange(E) % 16).float() / 4
    bias = torch.zeros(E)
    for scoring in ("sigmoid", "softmax"):
        if scoring == "softmax":    # half of the experts at 0, the bias picks from the other half
            w[16:, 0], w[16:, 1] = 0, 0
            bias = torch.where(torch.arange(E) < 16, torch.arange(E) + 2.0, -1.0)
        args = dict(scoring=scoring, renorm=renorm)
        idx, wt = moeq.moe_route_scored(x.bfloat16().cuda(), w.cuda(), k, bias=bias.cuda() if scoring == "softmax" else None,
                                        **args)
        ref, rw, _ = M.route_scored(x.double().numpy(), w.double().numpy(), k,
                                    bias=bias.double().numpy() if scoring == "softmax" else None, **args)
        np.testing.assert_array_equal(idx.cpu().numpy(), ref)
        # (not renormalised, a score below fp32's range is 0 or subnormal: 2^-149 apart)
        np.testing.assert_allclose(wt.cpu().numpy(), rw, rtol=1e-5, atol=0 if renorm else 2.0 ** -148)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("top", [30.0, 0.0, -7.5, -8.5, -20.0, -59.0, -61.0, -100.0, -400.0])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_weights_far_below_the_largest(scoring, top, T):
    """Picks down to e^-56 of the largest, whose own scores may leave fp32's
    range: each weight to fp32's precision.  The logits are exact in fp32; expf
    (2 ulp), the sums, two divisions and a rounding near 2^-126 (2e-7) stay
    below 2e-6, and l - top is exact."""
    E, k = 32, 8
    x = torch.zeros(T, 64)
    x[:, 0], x[:, 1] = 1, 0.25 * (1 + torch.arange(T) % 4)
    w = torch.zeros(E, 64)
    w[:, 0], w[:, 1] = top, -8.0 * torch.arange(E)
    w[k + 3:, 0] -= 200
    idx, wt = moeq.moe_route_scored(x.bfloat16().cuda(), w.cuda(), k, scoring=scoring)
    ref, rw, _ = M.route_scored(x.double().numpy(), w.double().numpy(), k, scoring=scoring)
    np.testing.assert_array_equal(idx.cpu().numpy(), ref)
    np.testing.assert_allclose(wt.cpu().numpy(), rw, rtol=1e-5, atol=0)


def check_picks(x, w, k, bias=None, rtol=1e-5, **kw):
    idx, wt = moeq.moe_route_scored(x.cuda(), w.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    ref, rw, _ = M.route_scored(x.double().numpy(), w.double().numpy(), k,
                                bias=None if bias is None else bias.double().numpy(), **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ref)
    np.testing.assert_allclose(wt.cpu().numpy(), rw, rtol=rtol, atol=1e-30)   # (RTOL of the scored router's tests)


@pytest.mark.parametrize("T", [1, 4, 33, 150])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,kept,top,k", [(256, 32, 7, 2, 8), (256, 32, 31, 1, 16), (256, 16, 3, 2, 16), (64, 32, 4, 2, 8),
                                            (32, 32, 9, 1, 9), (160, 32, 2, 1, 8), (96, 16, 16, 2, 5), (180, 20, 5, 2, 6),
                                            (99, 11, 4, 2, 7)])
def test_many_groups(E, G, kept, top, k, scoring, T):
    """Two lanes, and one, to a group; group counts that divide no warp."""
    g = torch.Generator().manual_seed(60 + G)
    x, w = torch.randn(T, 256, generator=g).bfloat16(), torch.randn(E, 256, generator=g) * 0.06
    b = torch.randn(E, generator=g) * 0.05
    kw = dict(scoring=scoring, n_groups=G, topk_groups=kept, group_top=top)
    check_picks(x, w, k, bias=b, **kw)
    check_picks(x, w, k, renorm=False, **kw)
    w = w[torch.arange(E) % 7]                   # ties inside groups and between them
    check_picks(x, w, k, **kw)
    check_picks(x, w, k, bias=torch.zeros(E), **kw)


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(256, 16), (256, 1), (48, 16), (16, 16)])
def test_all_experts_equal(E, k, scoring, T):
    """More experts tied at the cut than a warp has lanes."""
    x = torch.randn(T, 96, generator=torch.Generator().manual_seed(61)).bfloat16()
    w = torch.zeros(E, 96)
    for bias in (None, torch.zeros(E), torch.full((E,), 1e30), torch.full((E,), -1e30)):
        check_picks(x, w, k, bias=bias, scoring=scoring)
        check_picks(x, w, k, bias=bias, scoring=scoring, n_groups=4 if E >= 48 else 1, topk_groups=2 if E >= 48 else 1,
                    group_top=2)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_biases_out_of_range(scoring, T):
    g = torch.Generator().manual_seed(62)
    x, w = torch.randn(T, 128, generator=g).bfloat16(), torch.randn(40, 128, generator=g) * 0.1
    b = torch.randn(40, generator=g) * 0.05
    inf = float("inf")
    for places, value in (([3, 30], inf), ([3, 4, 30], 3e38), ([5, 6], float("nan")), ([0, 39], -3e38), (list(range(35)), -inf)):
        c = b.clone()
        c[places] = value
        for kw in (dict(), dict(n_groups=8, topk_groups=3, group_top=2), dict(n_groups=8, topk_groups=3)):
            check_picks(x, w, 6, bias=c, scoring=scoring, **kw)
    c = b.clone()
    c[3], c[4], c[20] = inf, -inf, float("nan")  # a group's sum is NaN, and counts as -inf
    check_picks(x, w, 6, bias=c, scoring=scoring, n_groups=8, topk_groups=3, group_top=2)
