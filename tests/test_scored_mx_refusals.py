"""What the scored router and the MXFP4 calls refuse, before any launch: the
C ABI's argument checks and the size functions (no GPU needed)."""
import pytest

from quantized_moe_expert_histogram_b200 import build, moeq

OK, INVALID, SHAPE, WORKSPACE = 0, 1, 2, 6
P = 4096  # an aligned address; no refused call looks at it


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moeq.open_library()


def route(L, T=4, d=256, E=64, k=8, scoring=1, groups=8, kept=4, top=2, x=P, w=P, idx=P, wt=P, ws=P, ws_bytes=1 << 30):
    return L.moe_route_scored(x, w, None, T, d, E, k, scoring, groups, kept, top, 1, 1.0, idx, wt, ws, ws_bytes, None, None)


@pytest.mark.parametrize("args,code,words", [
    (dict(T=-1), INVALID, "bad sizes"), (dict(d=0), INVALID, "bad sizes"), (dict(x=None), INVALID, "null"),
    (dict(idx=None), INVALID, "null"), (dict(k=65), SHAPE, "k <= E"), (dict(k=17), SHAPE, "k <= 16"),
    (dict(E=512, groups=8), SHAPE, "E <= 256"), (dict(d=250), SHAPE, "multiple of 32"), (dict(d=32800), SHAPE, "32768"),
    (dict(scoring=2), INVALID, "scoring"), (dict(groups=0), INVALID, "groups"), (dict(groups=7), INVALID, "groups"),
    (dict(kept=9), INVALID, "groups"), (dict(kept=0), INVALID, "groups"), (dict(top=3), INVALID, "groups"),
    (dict(groups=64, kept=64, top=1), SHAPE, "32 groups"), (dict(groups=8, kept=1, k=9), SHAPE, "k=9"),
    (dict(E=8, groups=8, kept=8), SHAPE, "group_top=2"), (dict(ws=None), WORKSPACE, "workspace"),
    (dict(ws_bytes=64), WORKSPACE, "workspace"), (dict(ws=P + 4), INVALID, "aligned"), (dict(x=P + 2), INVALID, "aligned"),
])
def test_route_scored_refuses(lib, args, code, words):
    assert route(lib, **args) == code
    assert words in lib.moe_last_error().decode()


def quantize(L, x=P, dtype=1, rows=4, K=64, ld=64, inv=None, k=1, codes=P, scales=P):
    return L.moe_mx_quantize(x, dtype, rows, K, ld, inv, k, codes, scales, None, None)


@pytest.mark.parametrize("args,code,words", [
    (dict(rows=-1), INVALID, "bad arg"), (dict(K=0), INVALID, "bad arg"), (dict(dtype=3), INVALID, "bad arg"),
    (dict(ld=32), INVALID, "bad arg"), (dict(k=0), INVALID, "bad arg"), (dict(k=2), INVALID, "inv_perm"),
    (dict(K=48), SHAPE, "multiple of 32"), (dict(ld=66), SHAPE, "16 bytes"), (dict(x=None), INVALID, "null"),
    (dict(codes=None), INVALID, "null"), (dict(x=P + 8), INVALID, "aligned"), (dict(codes=P + 4), INVALID, "aligned"),
    (dict(rows=1 << 30, inv=P, k=4), SHAPE, "2^31"),
])
def test_quantize_refuses(lib, args, code, words):
    assert quantize(lib, **args) == code
    assert words in lib.moe_last_error().decode()


def test_dequantize_and_pack_refuse(lib):
    assert lib.moe_mx_dequantize(P, P, 4, 64, 2, P, None) == INVALID      # fp16 does not hold every value
    assert lib.moe_mx_dequantize(P, P, 4, 48, 0, P, None) == SHAPE
    assert lib.moe_mx_dequantize(None, P, 4, 64, 0, P, None) == INVALID
    assert lib.moe_mx_pack(P, 0, 2, 100, 128, P, None, None) == SHAPE
    assert lib.moe_mx_pack(P, 9, 2, 128, 128, P, None, None) == INVALID
    assert lib.moe_mx_pack(P, 0, 2, 128, 128, None, None, None) == INVALID
    assert lib.moe_mx_pack_ffn(P, P, P, 0, 2, 128, 100, P, None, None) == SHAPE
    assert lib.moe_mx_pack_ffn(P, None, P, 0, 2, 128, 128, P, None, None) == INVALID


def gemm(L, rows=8, E=4, N=128, K=128, dtype=2, codes=P, scales=P, off=P, mats=P, out=P):
    return L.moe_mx_grouped_gemm(codes, scales, off, mats, rows, E, N, K, dtype, out, None, None)


def ffn(L, rows=8, E=4, d=128, F=128, ws=P, nbytes=1 << 20, codes=P, out=P):
    return L.moe_grouped_ffn_mx(codes, P, P, P, rows, E, d, F, ws, nbytes, out, None, None)


@pytest.mark.parametrize("args,code,words", [
    (dict(rows=-1), INVALID, "bad sizes"), (dict(N=0), INVALID, "bad sizes"), (dict(N=100), SHAPE, "128"),
    (dict(K=96), SHAPE, "128"), (dict(E=257), SHAPE, "256"), (dict(dtype=5), INVALID, "dtype"),
    (dict(codes=None), INVALID, "null"), (dict(off=None), INVALID, "null"), (dict(out=P + 2), INVALID, "aligned"),
    (dict(scales=P + 8), INVALID, "aligned"), (dict(rows=2 ** 31 - 1, N=1 << 24), SHAPE, "tiles"),
    # out of order, the offsets of 256 experts could claim all the rows 128 times
    (dict(rows=1 << 20, N=1 << 19, E=256), SHAPE, "tiles"),
])
def test_grouped_gemm_refuses(lib, args, code, words):
    assert gemm(lib, **args) == code
    assert words in lib.moe_last_error().decode()


def test_ffn_refuses(lib):
    assert ffn(lib, F=100) == SHAPE
    assert ffn(lib, d=100) == SHAPE
    assert ffn(lib, nbytes=16) == WORKSPACE
    assert ffn(lib, ws=None) == WORKSPACE
    assert ffn(lib, ws=P + 8) == INVALID
    assert ffn(lib, codes=None) == INVALID


def test_empty_calls_are_no_ops(lib):
    assert route(lib, T=0, x=None, w=None, idx=None, wt=None, ws=None, ws_bytes=0) == OK
    assert quantize(lib, rows=0, x=None, codes=None, scales=None) == OK
    assert lib.moe_mx_dequantize(None, None, 0, 64, 0, None, None) == OK
    assert gemm(lib, rows=0, codes=None, scales=None, off=None, mats=None, out=None) == OK
    assert lib.moe_grouped_ffn_mx(None, None, None, None, 0, 4, 128, 128, None, 0, None, None, None) == OK


def test_sizes(lib):
    assert lib.moe_mx_matrix_bytes(128, 256) == 128 * 256 * 17 // 32
    assert lib.moe_mx_blob_bytes(2048, 1024) == 3 * 2048 * 1024 * 17 // 32
    for N, K in ((0, 128), (128, 100), (-128, 128)):
        assert lib.moe_mx_matrix_bytes(N, K) == 0
    assert lib.moe_mx_blob_bytes(128, 64) == 0
    assert lib.moe_ffn_mx_workspace_bytes(3, 128) == 256 + 256
    assert lib.moe_ffn_mx_workspace_bytes(0, 128) == 256
    assert lib.moe_route_scored_workspace_bytes(0, 256, 64) >= 256
