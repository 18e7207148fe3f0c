"""MXFP4 products: tables that do not cover the rows; the FFN's two stages
apart, at sizes where a bound of the whole would say little."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as M
from quantized_moe_expert_histogram_b200 import build, moeq
from quantized_moe_expert_histogram_b200.layer import MxMoELayer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moeq.load()


def normal(*shape, seed=0, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("table,code", [([0, 3, 6], 0), ([2, 4, 6], moeq.DEV_BAD_INDEX), ([0, 2, 4], moeq.DEV_BAD_INDEX),
                                        ([0, 6, 4], moeq.DEV_BAD_INDEX), ([-1, 4, 6], moeq.DEV_BAD_INDEX)])
def test_a_table_that_does_not_cover_the_rows_is_flagged(table, code):
    """And the rows outside keep what they held."""
    rows, d, F = 6, 128, 128
    codes, scales = moeq.moe_mx_quantize(normal(rows, d, seed=1))
    mats = moeq.moe_mx_pack(normal(2, d, d, seed=2, std=0.1))
    blobs = moeq.moe_mx_pack_ffn(normal(2, F, d, seed=3), normal(2, F, d, seed=4), normal(2, d, F, seed=5))
    off = torch.tensor(table, dtype=torch.int32, device="cuda")
    head, tail = max(table[0], 0), max(table)
    st, out = status(), torch.full((rows, d), 9.0, device="cuda")
    moeq.moe_mx_grouped_gemm(codes, scales, off, mats, d, dtype=torch.float32, out=out, status=st)
    assert st.item() == code
    st, y = status(), torch.full((rows, d), 9.0, device="cuda", dtype=torch.float16)
    moeq.moe_grouped_ffn_mx(codes, scales, off, blobs, F, y_perm=y, status=st)
    assert st.item() == code
    for t in (out, y):
        assert (t[:head] == 9).all() and (t[tail:] == 9).all() and (t[head:tail] != 9).any(1).all()


@pytest.mark.parametrize("rows_of,d,F", [([400, 129, 0, 500, 1, 700], 2432, 1536), ([1, 0, 3, 140], 4096, 512),
                                         ([300, 17], 256, 4096), ([2], 128, 8192)])
def test_ffn_stages(rows_of, d, F):
    """hq from the workspace against the fp64 SwiGLU: equal, but for elements
    that lie within fp32's rounding of a rounding point (the sums before it
    are exact); then y against the product of that hq within its fp32 sum's
    bound and one rounding to fp16."""
    rng = np.random.default_rng(d + F)
    E, R = len(rows_of), sum(rows_of)
    x = M.exact_rows(rng, R, d)
    wg, wu = (M.exact_rows(rng, E * F, d, -8).reshape(E, F, d) for _ in range(2))
    wd = M.rounded(rng.standard_normal((E, d, F)) * 0.05)
    gpu = [torch.from_numpy(v).float().cuda() for v in (x, wg, wu, wd)]
    codes, scales = moeq.moe_mx_quantize(gpu[0])
    off = torch.tensor(np.concatenate([[0], np.cumsum(rows_of)]), dtype=torch.int32).cuda()
    ws, st = torch.empty(moeq.moe_ffn_mx_workspace_bytes(R, F), dtype=torch.uint8, device="cuda"), status()
    y = moeq.moe_grouped_ffn_mx(codes, scales, off, moeq.moe_mx_pack_ffn(*gpu[1:]), F, workspace=ws, status=st)
    assert st.item() == 0
    ws, y, o = ws.cpu().numpy(), y.double().cpu().numpy(), off.tolist()
    at = (R * (F // 2) + 255) // 256 * 256
    byte = ws[at:at + R * (F // 32)].reshape(R, F // 32)
    hq = M.values(M.unpack_codes(ws[:R * (F // 2)].reshape(R, F // 2)), byte)
    near = 0
    for e in range(E):
        r = slice(o[e], o[e + 1])
        if rows_of[e] == 0:
            continue
        q, lo, hi = M.hidden(x[r], wg[e], wu[e])
        near += (lo != hi).sum()
        assert ((hq[r] >= lo) & (hq[r] <= hi)).all()
        ref, tol = M.product(hq[r], wd[e])
        lim = tol + M.half_step(np.abs(ref) + tol, 2.0 ** -10, 2.0 ** -24)
        assert (np.abs(y[r] - ref) <= lim).all()
        # far below |y|: F 2^-23 times a sum of F magnitudes, beside a sum that is about its root
        assert np.median(lim) < (1.5 * F ** 1.5 * 2.0 ** -23 + 2.0 ** -9) * np.median(np.abs(ref))
    assert near < 1e-3 * hq.size


def test_empty_batches():
    """No tokens, no rows: outputs of no rows, from each call and the layer."""
    d, E, k, F = 256, 8, 2, 128
    blobs = moeq.moe_mx_pack_ffn(normal(E, F, d, seed=6), normal(E, F, d, seed=7), normal(E, d, F, seed=8))
    w = normal(E, d, seed=9)
    x = normal(4, d, seed=10, dtype=torch.bfloat16)
    idx, wt = moeq.moe_route_scored(x[:0], w, k)
    assert idx.shape == wt.shape == (0, k)
    codes, scales = moeq.moe_mx_quantize(x[:0], inv_perm=torch.empty(0, k, dtype=torch.int32, device="cuda"), k=k)
    assert codes.shape == (0, d // 2) and moeq.moe_mx_dequantize(codes, scales).shape == (0, d)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    assert moeq.moe_grouped_ffn_mx(codes, scales, off, blobs, F).shape == (0, d)
    assert moeq.moe_mx_grouped_gemm(codes, scales, off, moeq.moe_mx_pack(normal(E, 128, d, seed=11)), 128).shape == (0, 128)
    layer = MxMoELayer(d, E, k, F, w, blobs, 4)
    want = layer.forward(x).clone()
    assert layer.forward(x[:0]).shape == (0, d) and layer.buf["status"].item() == 0
    assert torch.equal(layer.forward(x), want)
