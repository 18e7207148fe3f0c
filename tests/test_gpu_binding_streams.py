"""Outputs and workspaces that a call makes for itself on another stream,
beside memory that other streams still use."""
import pytest
import torch

from quantized_moe_expert_histogram_b200 import build, moeq

pytestmark = pytest.mark.gpu

SLEEP = 200_000_000  # cycles: a tenth of a second of work queued on a stream


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moeq.load()


ROWS, K = 4096, 2048


def calls():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(ROWS, K, generator=g).bfloat16().cuda()
    w = (torch.randn(64, K, generator=g) * 0.02).cuda()
    mat = moeq.moe_mx_pack((torch.randn(1, K, K, generator=g) * 0.02).cuda())
    codes, scales = moeq.moe_mx_quantize(x)
    off = torch.tensor([0, ROWS], dtype=torch.int32, device="cuda")
    # each with the bytes of its largest output or workspace
    return {
        "quantize": (lambda s: moeq.moe_mx_quantize(x, stream=s)[0], ROWS * K // 2),
        "dequantize": (lambda s: moeq.moe_mx_dequantize(codes, scales, stream=s), ROWS * K * 2),
        "product": (lambda s: moeq.moe_mx_grouped_gemm(codes, scales, off, mat, K, stream=s), ROWS * K * 2),
        "route_scored": (lambda s: moeq.moe_route_scored(x, w, 8, stream=s)[1],
                         moeq.moe_route_scored_workspace_bytes(ROWS, K, 64)),
        "route_topk": (lambda s: moeq.moe_route_topk(x, w, None, 8, stream=s)[1], moeq.moe_route_workspace_bytes(ROWS, K, 64)),
    }


@pytest.mark.parametrize("name", ["quantize", "dequantize", "product", "route_scored", "route_topk"])
def test_memory_that_queued_work_still_reads_is_left_alone(name):
    call, nbytes = calls()[name]
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    src = [torch.full((nbytes,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    keep = [torch.empty_like(t) for t in src]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for a, b in zip(keep, src):
        a.copy_(b)
    del src, a, b                   # released with the copies still queued
    got = call(side)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in keep)
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", ["quantize", "dequantize", "product"])
def test_an_output_released_with_work_queued_is_not_given_out_again(name):
    call, nbytes = calls()[name]
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    keep = got.clone()
    del got
    with torch.cuda.stream(side):   # the side stream's next tensors of that size
        for _ in range(3):
            torch.full((nbytes,), 9, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(keep, want)
