"""Calls that are refused, or return, before any launch (no GPU needed)."""
import contextlib

import pytest
import torch

from quantized_moe_expert_histogram_b200 import moeq
from quantized_moe_expert_histogram_b200.layer import MxMoELayer


class Library:
    """Every size is 256 bytes, every call succeeds and is noted."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_bytes"):
                return 256
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    L = Library()
    monkeypatch.setattr(moeq, "load", lambda: L)
    monkeypatch.setattr(moeq, "_ptr", lambda *a, **k: 0)
    monkeypatch.setattr(moeq, "_stream", lambda s: 0)
    monkeypatch.setattr(moeq, "_on", lambda *a: contextlib.nullcontext())
    return L


def half(*shape):
    return torch.zeros(*shape, dtype=torch.float16)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.mark.parametrize("bad", [dict(residual=bf16(3, 64)), dict(y=bf16(3, 64)), dict(inv_perm=i32(7)), dict(y_perm=half(7, 64))])
def test_combine_refuses_tensors_it_would_run_past(lib, bad):
    args = dict(y_perm=half(8, 64), inv_perm=i32(8), topk_w=torch.zeros(4, 2), residual=bf16(4, 64), y=bf16(4, 64))
    moeq.moe_unpermute_combine(**args)
    assert lib.calls == ["moe_unpermute_combine"]
    with pytest.raises(ValueError, match=next(iter(bad))):
        moeq.moe_unpermute_combine(**{**args, **bad})
    assert len(lib.calls) == 1


@pytest.mark.parametrize("bad", [dict(residual=bf16(3, 64)), dict(y=bf16(3, 64))])
def test_ffn_combine_refuses_tensors_it_would_run_past(lib, bad):
    args = dict(x_perm=half(8, 64), offsets=i32(9), blobs=torch.zeros(8, 256, dtype=torch.uint8), T=4, k=2, E=8, d=64, F=64,
                group=64, layout=0, perm=i32(8), inv_perm=i32(8), topk_w=torch.zeros(4, 2))
    moeq.moe_grouped_ffn_combine(**args)
    with pytest.raises(ValueError, match=next(iter(bad))):
        moeq.moe_grouped_ffn_combine(**args, **bad)
    assert len(lib.calls) == 1


def test_layer_refuses_a_residual_of_another_shape(lib):
    layer = MxMoELayer(128, 8, 2, 128, torch.zeros(8, 128), torch.zeros(8, 256, dtype=torch.uint8), 16, device="cpu")
    for shape in ((3, 128), (1, 128), (128,), (4, 64)):
        with pytest.raises(ValueError, match="residual"):
            layer.forward(bf16(4, 128), residual=bf16(*shape))
    assert not lib.calls


def test_quantising_no_rows_needs_no_places():
    """An empty permutation has no address."""
    from quantized_moe_expert_histogram_b200 import build
    build.build()
    L = moeq.open_library()
    assert L.moe_mx_quantize(None, 1, 0, 64, 64, None, 4, None, None, None, None) == 0
    assert L.moe_mx_quantize(4096, 1, 4, 64, 64, None, 4, 4096, 4096, None, None) == 1
