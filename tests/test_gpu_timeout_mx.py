"""On-device failure detection of the MXFP4 product and of the scored
router's tensor-core logits, without a GPU fault: every wait is bounded.  The
test hook shortens the limit to 20 ms and has one warp withhold an arrive
that no copy stands behind; the launch returns, the status word carries
MOE_DEV_TIMEOUT, and the next call is what the one before it was."""
import pytest
import torch

from quantized_moe_expert_histogram_b200 import build, moeq

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _hooks():
    build.build()
    moeq.load()
    yield
    moeq.moe_debug_mx_timeout(0)


def normal(*shape, seed, std=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda() * std


def product():
    # 40 x 8 tiles of 128 rows x 256 outputs: CTA 0 has a second one
    codes, scales = moeq.moe_mx_quantize(normal(5120, 512, seed=1))
    mats = moeq.moe_mx_pack(normal(1, 2048, 512, seed=2, std=0.05))
    off = torch.tensor([0, 5120], dtype=torch.int32, device="cuda")
    return lambda st: [moeq.moe_mx_grouped_gemm(codes, scales, off, mats, 2048, status=st)]


def ffn():
    codes, scales = moeq.moe_mx_quantize(normal(5120, 256, seed=3))
    blobs = moeq.moe_mx_pack_ffn(normal(1, 1024, 256, seed=4, std=0.05), normal(1, 1024, 256, seed=5, std=0.05),
                                 normal(1, 256, 1024, seed=6, std=0.05))
    off = torch.tensor([0, 5120], dtype=torch.int32, device="cuda")
    return lambda st: [moeq.moe_grouped_ffn_mx(codes, scales, off, blobs, 1024, status=st)]


def route():
    # 32 x 2 tiles in two slices of four chunks
    x, w = normal(8191, 512, seed=7).bfloat16(), normal(256, 512, seed=8, std=0.02)
    return lambda st: list(moeq.moe_route_scored(x, w, 8, scoring="sigmoid", status=st))


@pytest.mark.parametrize("case", [product, ffn, route])
def test_bounded_waits_run_out_and_the_next_call_is_exact(case):
    call = case()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = call(st)
    assert st.item() == 0
    moeq.moe_debug_mx_timeout(1)
    call(st)                         # returns instead of hanging
    assert st.item() & moeq.DEV_TIMEOUT
    moeq.moe_debug_mx_timeout(0)
    st.zero_()
    got = call(st)
    assert st.item() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
