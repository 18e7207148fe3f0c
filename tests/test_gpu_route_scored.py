"""The scored router against the fp64 oracle: expert ids exactly (near and
exact ties, masks, groups, rows that are not finite), weights within the
error of fp32 logits; and the MXFP4 layer that starts with it."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import mx_oracle as M
from quantized_moe_expert_histogram_b200 import build, moeq
from quantized_moe_expert_histogram_b200.layer import MxMoELayer

pytestmark = pytest.mark.gpu

# Weights: a logit error dl moves a score (and, renormalised, a weight) by at
# most 2 |dl| relative.  The fp32 logits here (|l| <= 10, d <= 4096) err by
# less than 2e-6 (sums of 32 products: a few 1e-7 typically), fp32 exp,
# division and sums by a few 1e-7.
RTOL = 1e-5

ROUTERS = [dict(), dict(scoring="sigmoid"), dict(scoring="sigmoid", renorm=False, scale=2.5),
           dict(renorm=False), dict(bias=True), dict(scoring="sigmoid", bias=True, scale=2.5),
           dict(scoring="sigmoid", bias=True, n_groups=8, topk_groups=4, group_top=2),
           dict(scoring="sigmoid", n_groups=4, topk_groups=1, group_top=1),
           dict(bias=True, n_groups=8, topk_groups=3, group_top=2), dict(n_groups=2, topk_groups=1, group_top=2)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moeq.load()


def draw(T, d, E, seed, std=0.02):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, d, generator=g).bfloat16(), torch.randn(E, d, generator=g) * std, torch.randn(E, generator=g) * 0.05


def check(x, w, k, bias=None, rtol=RTOL, **kw):
    idx, wt = moeq.moe_route_scored(x.cuda(), w.cuda(), k, bias=None if bias is None else bias.cuda(), **kw)
    ref, rw, _ = M.route_scored(x.double().numpy(), w.double().numpy(), k,
                                bias=None if bias is None else bias.double().numpy(), **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), ref)
    np.testing.assert_allclose(wt.cpu().numpy(), rw, rtol=rtol, atol=1e-30)
    return ref


@pytest.mark.parametrize("router", range(len(ROUTERS)))
# one cluster launch (up to 8 tokens and 128 logits), tensor-core logits otherwise
@pytest.mark.parametrize("T,d,E,k", [(1, 2048, 64, 8), (8, 1088, 64, 8), (1, 512, 256, 8), (2, 576, 128, 5), (7, 256, 16, 2),
                                     (9, 2048, 64, 8), (3, 96, 64, 4), (127, 352, 96, 8), (130, 288, 128, 6), (300, 1024, 256, 8),
                                     (513, 224, 160, 8)])
def test_choice_and_weights(T, d, E, k, router):
    kw = dict(ROUTERS[router])
    x, w, b = draw(T, d, E, seed=100 + router)
    check(x, w, k, bias=b if kw.pop("bias", False) else None, **kw)


@pytest.mark.parametrize("T", [1, 33, 257])
@pytest.mark.parametrize("E,k,G", [(60, 4, 4), (8, 8, 1), (1, 1, 1), (40, 16, 5)])
def test_odd_expert_counts(T, E, k, G):
    x, w, b = draw(T, 64, E, seed=7, std=0.2)
    kept = G if G == 1 else G - 1
    for scoring in ("softmax", "sigmoid"):
        check(x, w, k, bias=b, scoring=scoring, n_groups=G, topk_groups=kept)


@pytest.mark.parametrize("T", [4, 40, 140])
@pytest.mark.parametrize("router", range(len(ROUTERS)))
def test_exact_ties_go_to_the_lower_index(router, T):
    kw = dict(ROUTERS[router])
    x, w, b = draw(T, 512, 64, seed=8)
    w = w[torch.arange(64) % 13]                # each row many times, across groups
    check(x, w, 8, bias=torch.zeros(64) if kw.pop("bias", False) else None, **kw)


@pytest.mark.parametrize("T", [6, 60, 150])
@pytest.mark.parametrize("router", range(len(ROUTERS)))
def test_near_ties(router, T):
    """Rows that differ in their last fp32 bits: closer than the fp32 sums'
    error, apart in fp64."""
    kw = dict(ROUTERS[router])
    x, w, b = draw(T, 1024, 64, seed=9)
    w = w[torch.arange(64) % 8].clone()
    w.view(torch.int32)[:, ::7] += torch.arange(64, dtype=torch.int32)[:, None] % 5
    check(x, w, 8, bias=b[torch.arange(64) % 8] if kw.pop("bias", False) else None, **kw)


@pytest.mark.parametrize("T", [3, 21, 129])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,kept,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_masked_experts(scoring, G, kept, top, T):
    x, w, b = draw(T, 256, 32, seed=10)
    kw = dict(scoring=scoring, n_groups=G, topk_groups=kept, group_top=top)
    b[[0, 3, 9, 17, 30]] = -float("inf")
    ref = check(x, w, 4, bias=b, **kw)
    assert not np.isin(ref, [0, 3, 9, 17, 30]).any()
    b[:] = -float("inf")                        # nothing left: the lowest indexes
    assert (check(x, w, 4, bias=b, **kw) == np.arange(4)).all()
    b[[11, 20]] = 0.1                           # fewer left than k
    check(x, w, 4, bias=b, **kw)
    b[12] = float("nan")
    check(x, w, 4, bias=b, **kw)


@pytest.mark.parametrize("T", [6, 20, 131])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_rows_that_are_not_finite(scoring, bias, T):
    x, w, b = draw(T, 128, 16, seed=11)
    x[1, 5] = float("inf")
    x[2, 5] = float("nan")
    x[3, 7], x[3, 8] = float("inf"), -float("inf")
    x[4] = 3e38                                 # overflows fp32, not fp64
    w[3] = 0
    for G, kept, top in ((1, 1, 1), (4, 2, 2)):
        check(x, w, 3, bias=b if bias else None, scoring=scoring, n_groups=G, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("T", [2, 12, 140])
def test_far_scores(T):
    """Sigmoid scores that leave fp32's range, and saturated ones."""
    x, w, b = draw(T, 256, 32, seed=12)
    x[:, 0] = 1.0
    w[:, 0] = -120.0
    # scores of about e^-120: the logits' fp32 rounding (120 x 2^-24 x a few) is what the weights show
    check(x, w, 4, scoring="sigmoid", rtol=2e-4)
    check(x, w, 4, scoring="sigmoid", bias=b, rtol=2e-4)
    w[:, 0] = 30.0
    check(x, w, 4, scoring="sigmoid", bias=b)


@pytest.mark.parametrize("T,d,E", [(200, 2048, 256), (64, 1024, 64)])
def test_logit_bounds_hold(T, d, E):
    """Weights of very different magnitudes along a row, sums that cancel:
    the choice stays that of the fp64 scores (it would not if the error
    bounds were too small)."""
    x, w, _ = draw(T, d, E, seed=14)
    w = w * torch.exp2(torch.randint(-12, 8, (1, d), generator=torch.Generator().manual_seed(15)).float())
    x[:, 1::2] = x[:, 0::2]
    w[:, 1::2] = -w[:, 0::2] * (1 + 2.0 ** -12 * torch.randn(E, d // 2, generator=torch.Generator().manual_seed(16)))
    for kw in (dict(), dict(scoring="sigmoid"), dict(scoring="sigmoid", bias=torch.linspace(-1e-4, 1e-4, E)),
               dict(scoring="sigmoid", n_groups=8, topk_groups=3, group_top=2)):
        # sums of terms of magnitude about 2^7 that cancel to about 1e-2: relative to the
        # weights, fp32's rounding shows
        check(x, w, 8, rtol=2e-2, **kw)


@pytest.mark.parametrize("T", [4, 60, 200])
def test_subnormal_and_huge_magnitudes(T):
    """Weights whose lower bf16 parts are subnormal, activations that are, and
    rows of very large ones."""
    x, w, b = draw(T, 128, 32, seed=17)
    scale = torch.exp2(torch.linspace(-120, 120, T)).bfloat16()[:, None]
    x = x * scale
    for ws in (2.0 ** -110, 1.0, 2.0 ** 6):
        for kw in (dict(), dict(scoring="sigmoid", bias=b), dict(scoring="sigmoid", n_groups=4, topk_groups=2)):
            # logits up to 2^120: where they are far apart in fp32's rounding the softmax's weights show it
            idx, _ = moeq.moe_route_scored(x.cuda(), (w * ws).cuda(), 4, **{k: v.cuda() if k == "bias" else v for k, v in kw.items()})
            ref, _, _ = M.route_scored(x.double().numpy(), (w * ws).double().numpy(), 4,
                                       **{k: v.double().numpy() if k == "bias" else v for k, v in kw.items()})
            np.testing.assert_array_equal(idx.cpu().numpy(), ref)


def test_calls_on_two_streams_at_once():
    """Two streams, no order between them, workspaces and outputs allocated by
    the calls: each gives what it gives alone."""
    args = [tuple(t.cuda() for t in draw(300, 512, 64, seed=20 + i)) for i in range(2)]
    want = [moeq.moe_route_scored(x, w, 4, bias=b, scoring="sigmoid") for x, w, b in args]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, (x, w, b) in enumerate(args):
            got[i].append(moeq.moe_route_scored(x, w, 4, bias=b, scoring="sigmoid", stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for idx, wt in got[i]:
            assert torch.equal(idx, want[i][0]) and torch.equal(wt, want[i][1])


def test_workspace_of_the_largest_batch_serves_the_smaller():
    for d, E in ((256, 64), (2048, 256), (64, 8)):
        sizes = [moeq.moe_route_scored_workspace_bytes(T, d, E) for T in (1, 7, 8, 100, 127, 128, 129, 1000, 4096, 5000, 70000)]
        assert sizes == sorted(sizes)


def test_outputs_workspace_and_refusals():
    x, w, b = (t.cuda() for t in draw(50, 512, 64, seed=13))
    idx = torch.full((52, 4), -7, dtype=torch.int32, device="cuda")
    wt = torch.full((52, 4), -7.0, device="cuda")
    ws = torch.empty(moeq.moe_route_scored_workspace_bytes(50, 512, 64), dtype=torch.uint8, device="cuda")
    a = moeq.moe_route_scored(x, w, 4, bias=b, scoring="sigmoid", topk_idx=idx[:50], topk_w=wt[:50], workspace=ws)
    c = moeq.moe_route_scored(x, w, 4, bias=b, scoring="sigmoid")
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    assert (idx[50:] == -7).all() and (wt[50:] == -7).all()
    with pytest.raises(ValueError):
        moeq.moe_route_scored(x, w, 4, scoring="relu")
    with pytest.raises(ValueError):
        moeq.moe_route_scored(x, w, 4, bias=b[:3])
    with pytest.raises(ValueError):
        moeq.moe_route_scored(x, w.cpu(), 4)
    with pytest.raises(TypeError):
        moeq.moe_route_scored(x.float(), w, 4)
    with pytest.raises(moeq.MoeError) as err:
        moeq.moe_route_scored(x, w, 4, workspace=ws[:64])
    assert err.value.code == 6
    assert moeq.moe_route_scored(x[:0], w, 4)[0].shape == (0, 4)


# ---- the layer -------------------------------------------------------------------------

def layer_case(T, d, E, k, F, seed, **routing):
    x, wr, b = draw(T, d, E, seed)
    g = torch.Generator().manual_seed(seed + 1)
    wg, wu, wd = (torch.randn(E, *s, generator=g) * 0.05 for s in ((F, d), (F, d), (d, F)))
    layer = MxMoELayer.from_weights(wr.cuda(), wg.cuda(), wu.cuda(), wd.cuda(), k, T + 3, bias=b.cuda(), **routing)
    return x, wr, b, (wg, wu, wd), layer


@pytest.mark.parametrize("T,residual", [(1, False), (5, True), (40, True)])
def test_layer_against_the_oracle(T, residual):
    d, E, k, F = 256, 16, 4, 128
    routing = dict(scoring="sigmoid", n_groups=4, topk_groups=2, group_top=2, scale=2.5)
    x, wr, b, ws, layer = layer_case(T, d, E, k, F, 200 + T, **routing)
    res = torch.randn(T, d, generator=torch.Generator().manual_seed(1)).bfloat16() if residual else None
    y = layer.forward(x.cuda(), residual=None if res is None else res.cuda()).double().cpu().numpy()
    v = layer.views(T)
    assert v["status"].item() == 0
    idx, wt, _ = M.route_scored(x.double().numpy(), wr.double().numpy(), k, bias=b.double().numpy(), **routing)
    np.testing.assert_array_equal(v["topk_idx"].cpu().numpy(), idx)
    counts, offsets, perm, inv = O.permute(idx.reshape(-1), E)
    np.testing.assert_array_equal(v["offsets"].cpu().numpy(), offsets)
    np.testing.assert_array_equal(v["inv_perm"].cpu().numpy(), inv)
    xq = M.rounded(x.double().numpy())
    ref = np.zeros((T, d)) if res is None else res.double().numpy()
    lim = np.abs(ref) * 1e-6
    q = [M.rounded(w.double().numpy()) for w in ws]
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            ye, tol = M.ffn(xq[t:t + 1], q[0][e], q[1][e], q[2][e])
            ref[t] += wt[t, j] * ye[0]
            # y_perm's half step in fp16, the weight's error, the fp32 sum
            lim[t] += wt[t, j] * (tol[0] + (np.abs(ye[0]) + tol[0]) * (2.0 ** -11 + RTOL + 1e-6) + 2.0 ** -25)
    err = np.abs(y - ref)
    assert (err <= lim + (np.abs(ref) + lim) * 2.0 ** -8).all(), (err / lim).max()


def test_layer_in_a_graph_and_on_another_stream():
    x, wr, b, ws, layer = layer_case(24, 256, 16, 2, 128, 300, scoring="sigmoid")
    x = x.cuda()
    want = layer.forward(x).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    layer.buf["y"].zero_()
    s.wait_stream(torch.cuda.current_stream())
    y = layer.forward(x, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer.forward(x)
    x2 = draw(24, 256, 16, 301)[0].cuda()
    x.copy_(x2)
    g.replay()
    got = y.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, layer.forward(x2))
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(28, 256, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("T,d,E", [(9, 4096, 200), (33, 96, 256), (700, 256, 256), (1500, 64, 72)])
@pytest.mark.parametrize("open_tokens", ["all", "some"])
def test_softmax_with_bias_by_fp64_rows(T, d, E, open_tokens):
    """Tokens whose choice hangs on the softmax's denominator: all of them
    (every expert twice), or those whose two best lie nearly together."""
    x, w, b = draw(T, d, E, seed=31, std=0.5 / d ** 0.5)
    if open_tokens == "all":
        w[E // 2:], b[E // 2:] = w[:E // 2], b[:E // 2]
    else:
        b *= 1e-3
    check(x, w, 7, bias=b)
    check(x, w, 7, bias=b, n_groups=4, topk_groups=2, group_top=2, renorm=False)
    a = moeq.moe_route_scored(x.cuda(), w.cuda(), 7, bias=b.cuda())
    c = moeq.moe_route_scored(x.cuda(), w.cuda(), 7, bias=b.cuda())
    assert all(torch.equal(p, q) for p, q in zip(a, c))


def test_softmax_with_bias_replayed():
    """The list of open tokens starts anew in every replay."""
    x, w, b = draw(90, 256, 64, seed=41)
    w[32:], b[32:] = w[:32], b[:32]             # every token is open
    xs, wd, bd = x.cuda(), w.cuda(), b.cuda()
    moeq.moe_route_scored(xs, wd, 4, bias=bd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, wt = moeq.moe_route_scored(xs, wd, 4, bias=bd)
    for seed in (42, 43):
        x = draw(90, 256, 64, seed=seed)[0]
        xs.copy_(x)
        g.replay()
        want = moeq.moe_route_scored(x.cuda(), wd, 4, bias=bd)
        assert torch.equal(idx, want[0]) and torch.equal(wt, want[1])


def test_layer_refuses_tensors_elsewhere():
    x, wr, b, ws, layer = layer_case(4, 256, 16, 2, 128, 301)
    with pytest.raises(ValueError, match="MxMoELayer.forward"):
        layer.forward(x)
