"""MXFP4 on the GPU against the fp64 oracle: quantisation and packing bit for
bit, the grouped product and the expert FFN within bounds derived from their
roundings (exact products, fp32 sums, one rounding of the output)."""
import numpy as np
import pytest
import torch

from oracle import mx_oracle as M
from quantized_moe_expert_histogram_b200 import build, moeq

pytestmark = pytest.mark.gpu

NP = {torch.float32: (2.0 ** -23, 2.0 ** -149), torch.bfloat16: (2.0 ** -7, 2.0 ** -133),
      torch.float16: (2.0 ** -10, 2.0 ** -24)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moeq.load()


def f64(t):
    return t.double().cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def normal(*shape, seed=0, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def table(rows_of):
    """offsets of the given rows per expert."""
    return torch.tensor(np.concatenate([[0], np.cumsum(rows_of)]), dtype=torch.int32).cuda()


def check_rows(x, codes, scales):
    code, byte = M.quantize(f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), byte)
    np.testing.assert_array_equal(codes.cpu().numpy(), M.pack_codes(code))


@pytest.mark.parametrize("dtype", list(NP))
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (5, 1056), (64, 2048), (1000, 256)])
def test_quantize_rows(rows, K, dtype):
    x = normal(rows, K, seed=rows) * torch.exp2(torch.linspace(-12, 12, rows, device="cuda"))[:, None]
    x = x.to(dtype)
    check_rows(x, *moeq.moe_mx_quantize(x))


def test_quantize_rounding_points_and_extremes():
    v = torch.zeros(8, 32)
    v[0, :8] = torch.tensor(M.GRID)
    v[0, 8:15] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    v[1] = -v[0]
    v[2, 0], v[2, 1] = 7.99, -7.5                # saturate
    v[3, :3] = torch.tensor([2.0 ** -140, 2.0 ** -149, -2.0 ** -130])   # subnormal
    v[4, :2] = torch.tensor([3.3e38, -1e38])
    v[5] = -0.0
    v[6, :4] = torch.tensor([1.5 * 2.0 ** -126, 2.0 ** -126, -2.0 ** -127, 2.0 ** -128])
    v[7] = torch.linspace(-6, 6, 32)
    x = v.cuda()
    st = status()
    codes, scales = moeq.moe_mx_quantize(x, status=st)
    check_rows(x, codes, scales)
    assert st.item() == 0
    want = M.values(*M.quantize(f64(x)))
    np.testing.assert_array_equal(f64(moeq.moe_mx_dequantize(codes, scales, dtype=torch.float32)), want)
    np.testing.assert_array_equal(f64(moeq.moe_mx_dequantize(codes, scales)), want)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_quantize_non_finite_blocks(value):
    x = normal(3, 96, seed=4)
    x[1, 40] = value
    st = status()
    codes, scales = moeq.moe_mx_quantize(x, status=st)
    assert st.item() == moeq.DEV_RANGE
    assert scales[1, 1].item() == 255 and (scales != 255).sum().item() == 8
    y = moeq.moe_mx_dequantize(codes, scales, dtype=torch.float32)
    assert torch.isnan(y[1, 32:64]).all() and torch.isnan(y).sum().item() == 32


def test_every_code_and_scale_dequantizes():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :16 * 16].cuda()   # 256 rows x 512 elements
    scales = torch.arange(256, dtype=torch.uint8).cuda()[:, None].repeat(1, 16).contiguous()
    want = M.values(M.unpack_codes(codes.cpu().numpy()), scales.cpu().numpy())
    # 4 and 6 times 2^126 or 2^127, and 2, 3 times 2^127, are 2^128 or more: no finite fp32 or bf16 (Inf)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32)
    assert (np.isinf(want).sum(axis=1)[:253] == 0).all()
    for dtype in (torch.float32, torch.bfloat16):
        np.testing.assert_array_equal(f64(moeq.moe_mx_dequantize(codes, scales, dtype=dtype)), want)


@pytest.mark.parametrize("T,k,K", [(1, 8, 64), (7, 2, 1024), (33, 4, 2080)])
def test_quantize_in_expert_order(T, k, K):
    x = normal(T, K, seed=5, dtype=torch.bfloat16)
    inv = torch.randperm(T * k, generator=torch.Generator().manual_seed(6)).int().cuda()
    codes, scales = moeq.moe_mx_quantize(x, inv_perm=inv.view(T, k), k=k)
    source = torch.empty(T * k, dtype=torch.long)
    source[inv.cpu().long()] = torch.arange(T * k) // k
    check_rows(x[source.cuda()], codes, scales)


def test_quantize_bad_places_are_skipped():
    x = normal(2, 64, seed=7)
    inv = torch.tensor([[0, 4], [-1, 3]], dtype=torch.int32, device="cuda")
    codes = torch.full((4, 32), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((4, 2), 7, dtype=torch.uint8, device="cuda")
    st = status()
    moeq.moe_mx_quantize(x, inv_perm=inv, k=2, codes=codes, scales=scales, status=st)
    assert st.item() == moeq.DEV_BAD_INDEX
    check_rows(x[[0, 1]], codes[[0, 3]], scales[[0, 3]])
    assert (codes[1:3] == 7).all() and (scales[1:3] == 7).all()   # rows no place names


def test_quantize_strided_rows():
    big = normal(9, 256, seed=8, dtype=torch.bfloat16)
    x = big[:, 64:192]
    check_rows(x, *moeq.moe_mx_quantize(x))
    with pytest.raises(ValueError):
        moeq.moe_mx_quantize(big.t())
    with pytest.raises(ValueError):
        moeq.moe_mx_quantize(x.cpu())
    with pytest.raises(TypeError):
        moeq.moe_mx_quantize(x.double())


@pytest.mark.parametrize("dtype", list(NP))
def test_pack(dtype):
    w = normal(2, 256, 384, seed=9, std=0.02, dtype=dtype)
    mats = moeq.moe_mx_pack(w)
    for e in range(2):
        np.testing.assert_array_equal(mats[e].cpu().numpy(), M.matrix(f64(w[e])))


def test_pack_ffn():
    d, F = 128, 256
    wg, wu, wd = (normal(2, *s, seed=10 + i, std=0.02) for i, s in enumerate(((F, d), (F, d), (d, F))))
    blobs = moeq.moe_mx_pack_ffn(wg, wu, wd)
    for e in range(2):
        np.testing.assert_array_equal(blobs[e].cpu().numpy(), M.ffn_blob(f64(wg[e]), f64(wu[e]), f64(wd[e])))


# ---- grouped product ---------------------------------------------------------------

ROWS = [[1], [0, 1, 0], [3, 0, 130, 17], [128, 256, 1, 127], [0, 0, 5]]


def gemm_case(rows_of, N, K, dtype, seed=20, spread=4):
    E, R = len(rows_of), int(sum(rows_of))
    # scales over a few octaves from block to block, in rows and weights
    x = normal(R, K, seed=seed) * torch.exp2(normal(R, K // 32, seed=seed + 1, std=spread / 4)).repeat_interleave(32, 1)
    w = normal(E, N, K, seed=seed + 2, std=0.05) * torch.exp2(
        normal(E, N, K // 32, seed=seed + 3, std=spread / 4)).repeat_interleave(32, 2)
    codes, scales = moeq.moe_mx_quantize(x)
    mats = moeq.moe_mx_pack(w)
    st = status()
    y = moeq.moe_mx_grouped_gemm(codes, scales, table(rows_of), mats, N, dtype=dtype, status=st)
    xq, wq = M.rounded(f64(x)), M.rounded(f64(w))
    o = np.concatenate([[0], np.cumsum(rows_of)])
    eps, tiny = NP[dtype]
    assert st.item() == 0
    got = f64(y)
    for e in range(E):
        ref, tol = M.product(xq[o[e]:o[e + 1]], wq[e])
        err = np.abs(got[o[e]:o[e + 1]] - ref)
        assert (err <= tol + M.half_step(np.abs(ref) + tol, eps, tiny)).all(), (e, err.max())


@pytest.mark.parametrize("dtype", list(NP))
@pytest.mark.parametrize("rows_of", ROWS)
@pytest.mark.parametrize("N,K", [(128, 128), (256, 512), (384, 896)])
def test_grouped_gemm(rows_of, N, K, dtype):
    gemm_case(rows_of, N, K, dtype)


@pytest.mark.parametrize("rows_of,N,K", [
    ([300] * 8, 2048, 128),                 # 128 outputs a tile
    ([200] * 64, 384, 256),                 # 256 outputs a tile, the last one half
    ([1300, 5, 0, 700], 2560, 1152),        # 256 outputs a tile, several row tiles, half a last K stage
    ([2] * 100, 128, 2048),
    ([300] * 12, 2048, 384),                # full and short row tiles, half a last K stage
    ([700, 0, 1, 900], 3456, 640),          # the last 128 outputs alone, one row, no row
    ([2600], 2048, 2304),                   # many stages
])
def test_grouped_gemm_tiles(rows_of, N, K):
    gemm_case(rows_of, N, K, torch.float16, seed=30)


def test_grouped_gemm_row_past_the_last_expert_stay():
    codes, scales = moeq.moe_mx_quantize(normal(6, 128, seed=40))
    mats = moeq.moe_mx_pack(normal(2, 128, 128, seed=41, std=0.1))
    out = torch.full((6, 128), 9.0, device="cuda")
    st = status()
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    moeq.moe_mx_grouped_gemm(codes, scales, off, mats, 128, dtype=torch.float32, out=out, status=st)
    assert st.item() == moeq.DEV_BAD_INDEX          # the table does not cover the rows
    assert (out[4:] == 9).all() and (out[:4] != 9).any()
    st = status()
    off = torch.tensor([0, 2, 1 << 20], dtype=torch.int32, device="cuda")
    y = moeq.moe_mx_grouped_gemm(codes, scales, off, mats, 128, dtype=torch.float32, status=st)
    assert st.item() == moeq.DEV_BAD_INDEX
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    assert torch.equal(y, moeq.moe_mx_grouped_gemm(codes, scales, off, mats, 128, dtype=torch.float32))


def test_grouped_gemm_nan_blocks_and_range():
    x = normal(5, 256, seed=42)
    x[2, 100] = float("nan")
    codes, scales = moeq.moe_mx_quantize(x)
    w = normal(1, 128, 256, seed=43)
    w[0, 7, 3] = float("inf")
    mats = moeq.moe_mx_pack(w)
    y = moeq.moe_mx_grouped_gemm(codes, scales, table([5]), mats, 128, dtype=torch.float32)
    nan = torch.isnan(y)
    assert nan[2].all() and nan[:, 7].all()
    nan[2], nan[:, 7] = False, False
    assert not nan.any()
    st = status()
    big, s = moeq.moe_mx_quantize(normal(3, 128, seed=44) * 1e4)
    moeq.moe_mx_grouped_gemm(big, s, table([3]), moeq.moe_mx_pack(normal(1, 128, 128, seed=45)), 128, status=st)
    assert st.item() == moeq.DEV_RANGE


# ---- expert FFN ----------------------------------------------------------------------

def ffn_weights(E, d, F, seed=50):
    return tuple(normal(E, *s, seed=seed + i, std=0.05) for i, s in enumerate(((F, d), (F, d), (d, F))))


@pytest.mark.parametrize("rows_of,d,F", [([1], 128, 128), ([0, 3, 0, 140], 256, 384), ([9, 128, 1], 384, 256),
                                         ([1, 1, 0, 2, 1, 1, 1, 1], 512, 512), ([260] * 12, 256, 2048),
                                         # 256 outputs a tile in both products
                                         ([400, 129, 0, 500, 1, 700], 2432, 1536)])
def test_ffn(rows_of, d, F):
    E, R = len(rows_of), int(sum(rows_of))
    wg, wu, wd = ffn_weights(E, d, F)
    x = normal(R, d, seed=60, dtype=torch.bfloat16)
    codes, scales = moeq.moe_mx_quantize(x)
    st = status()
    y = f64(moeq.moe_grouped_ffn_mx(codes, scales, table(rows_of), moeq.moe_mx_pack_ffn(wg, wu, wd), F, status=st))
    assert st.item() == 0
    o = np.concatenate([[0], np.cumsum(rows_of)])
    xq = M.rounded(f64(x))
    for e in range(E):
        if rows_of[e] == 0:
            continue
        ref, tol = M.ffn(xq[o[e]:o[e + 1]], *(M.rounded(f64(w[e])) for w in (wg, wu, wd)))
        err = np.abs(y[o[e]:o[e + 1]] - ref)
        lim = tol + M.half_step(np.abs(ref) + tol, *NP[torch.float16])
        assert (err <= lim).all(), (e, (err / lim).max())


def test_calls_repeat_bit_for_bit_and_in_a_graph():
    rows_of, d, F = [3, 0, 150, 9], 256, 256
    R = sum(rows_of)
    blobs = moeq.moe_mx_pack_ffn(*ffn_weights(4, d, F, seed=70))
    off = table(rows_of)
    x = normal(R, d, seed=71, dtype=torch.bfloat16)
    codes, scales = moeq.moe_mx_quantize(x)
    ws = torch.empty(moeq.moe_ffn_mx_workspace_bytes(R, F), dtype=torch.uint8, device="cuda")
    first = moeq.moe_grouped_ffn_mx(codes, scales, off, blobs, F)
    y = torch.zeros_like(first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            moeq.moe_mx_quantize(x, codes=codes, scales=scales)
            moeq.moe_grouped_ffn_mx(codes, scales, off, blobs, F, workspace=ws, y_perm=y)
    torch.cuda.current_stream().wait_stream(s)
    for seed in (71, 72):
        x.copy_(normal(R, d, seed=seed, dtype=torch.bfloat16))
        g.replay()
        torch.cuda.synchronize()
        again = moeq.moe_grouped_ffn_mx(*moeq.moe_mx_quantize(x), off, blobs, F)
        assert torch.equal(y, again)
    x.copy_(normal(R, d, seed=71, dtype=torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)


def test_binding_refusals():
    codes, scales = moeq.moe_mx_quantize(normal(4, 128, seed=80))
    mats = moeq.moe_mx_pack(normal(2, 128, 128, seed=81))
    off = table([2, 2])
    with pytest.raises(ValueError):
        moeq.moe_mx_grouped_gemm(codes, scales[:, :2], off, mats, 128)
    with pytest.raises(ValueError):
        moeq.moe_mx_grouped_gemm(codes, scales, off[:2], mats, 128)
    with pytest.raises(ValueError):
        moeq.moe_mx_grouped_gemm(codes, scales, off, mats, 256)
    with pytest.raises(moeq.MoeError) as err:
        moeq.moe_mx_grouped_gemm(codes, scales, off, mats, 130)
    assert err.value.code == 2
    with pytest.raises(TypeError):
        moeq.moe_mx_grouped_gemm(codes, scales, off.long(), mats, 128)
    with pytest.raises(ValueError):
        moeq.moe_mx_quantize(normal(4, 128), inv_perm=torch.zeros(3, dtype=torch.int32, device="cuda"), k=2)
