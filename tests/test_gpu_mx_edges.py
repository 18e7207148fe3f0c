"""MXFP4 products: tables that do not cover the rows."""
import pytest
import torch

from quantized_moe_expert_histogram_b200 import build, moeq

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
