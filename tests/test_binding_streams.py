"""Where the bindings' own outputs and workspaces come from when a call runs
on another stream (no GPU needed: the library, the streams and the pointers
are stand-ins, the allocations are CPU tensors)."""
import contextlib

import pytest
import torch

from quantized_moe_expert_histogram_b200 import moeq

T, D, E, K, F = 4, 128, 8, 2, 128


class Library:
    """Every size is 256 bytes, every call succeeds."""

    def __getattr__(self, name):
        return lambda *a: 256 if name.endswith("_bytes") else 0


class Allocations:
    def __init__(self, monkeypatch):
        self.current, self.made, self.recorded = "current", [], []

        @contextlib.contextmanager
        def on(stream):
            before, self.current = self.current, stream
            yield
            self.current = before

        def new_empty(t, shape, **kw):
            return self.note(t.new_zeros(shape, **kw))

        empty = torch.empty
        monkeypatch.setattr(moeq, "load", lambda: Library())
        monkeypatch.setattr(moeq, "_check", lambda fn, code: None)
        monkeypatch.setattr(moeq, "_ptr", lambda *a, **k: 0)
        monkeypatch.setattr(moeq, "_stream", lambda s: 0)
        monkeypatch.setattr(moeq, "_on", lambda *a: contextlib.nullcontext())
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(torch.Tensor, "new_empty", new_empty)
        monkeypatch.setattr(torch, "empty", lambda *a, **k: self.note(empty(*a, **k)))
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.recorded.append((id(t), s)))

    def note(self, t):
        self.made.append((t, self.current))
        return t


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


X, W, IDX = bf16(T, D), torch.zeros(E, D), i32(T, K)
ROWS = T * K
CALLS = {
    "moe_quant_pack": lambda s: moeq.moe_quant_pack(torch.zeros(E, F, D), torch.zeros(E, F, D), torch.zeros(E, D, F), 64, 0, stream=s),
    "moe_route_topk": lambda s: moeq.moe_route_topk(X, W, None, K, stream=s),
    "moe_route_topk_noalloc": lambda s: moeq.moe_route_topk_noalloc(X, W, None, K, stream=s),
    "moe_permute": lambda s: moeq.moe_permute(IDX, E, x=X, stream=s),
    "moe_route_permute": lambda s: moeq.moe_route_permute(X, W, None, K, w_bit=torch.zeros(E, 3, D), stream=s),
    "moe_static_bits": lambda s: moeq.moe_static_bits(IDX, u8(E), E, stream=s),
    "moe_bit_gate": lambda s: moeq.moe_bit_gate(X, torch.zeros(E, 3, D), None, IDX, stream=s),
    "moe_grouped_ffn_combine": lambda s: moeq.moe_grouped_ffn_combine(
        torch.zeros(ROWS, D).half(), i32(E + 1), u8(E, 16), T, K, E, D, F, 64, 0, i32(ROWS), i32(ROWS), torch.zeros(T, K), stream=s),
    "moe_grouped_ffn_wq": lambda s: moeq.moe_grouped_ffn_wq(torch.zeros(ROWS, D).half(), i32(E + 1), u8(E, 16), T, E, D, F, 64, 0, stream=s),
    "moe_unpermute_combine": lambda s: moeq.moe_unpermute_combine(torch.zeros(ROWS, D).half(), i32(ROWS), torch.zeros(T, K), stream=s),
    "moe_route_scored": lambda s: moeq.moe_route_scored(X, W, K, stream=s),
    "moe_mx_quantize": lambda s: moeq.moe_mx_quantize(X, stream=s),
    "moe_mx_dequantize": lambda s: moeq.moe_mx_dequantize(u8(T, D // 2), u8(T, D // 32), stream=s),
    "moe_mx_pack": lambda s: moeq.moe_mx_pack(torch.zeros(E, 128, D), stream=s),
    "moe_mx_pack_ffn": lambda s: moeq.moe_mx_pack_ffn(torch.zeros(E, F, D), torch.zeros(E, F, D), torch.zeros(E, D, F), stream=s),
    "moe_mx_grouped_gemm": lambda s: moeq.moe_mx_grouped_gemm(u8(T, D // 2), u8(T, D // 32), i32(E + 1), u8(E, 256), 128, stream=s),
    "moe_grouped_ffn_mx": lambda s: moeq.moe_grouped_ffn_mx(u8(T, D // 2), u8(T, D // 32), i32(E + 1), u8(E, 256), F, stream=s),
}


def tensors(v):
    if isinstance(v, torch.Tensor):
        return [v]
    return [t for x in (v.values() if isinstance(v, dict) else v if isinstance(v, tuple) else ()) for t in tensors(x)]


@pytest.mark.parametrize("name", CALLS)
def test_allocations_belong_to_the_call_stream(name, monkeypatch):
    """Made in the pool of the stream that the kernels run on, and what is
    returned is recorded as in use on the caller's."""
    a = Allocations(monkeypatch)
    out = tensors(CALLS[name]("side"))
    assert a.made and all(s == "side" for _, s in a.made)
    returned = {id(t) for t, _ in a.made} & {id(t) for t in out}
    assert returned and set(a.recorded) == {(i, "current") for i in returned}
    assert a.current == "current"


@pytest.mark.parametrize("stream", [None, "current"])
@pytest.mark.parametrize("name", CALLS)
def test_allocations_on_the_current_stream(name, stream, monkeypatch):
    a = Allocations(monkeypatch)
    CALLS[name](stream)
    assert a.made and all(s == "current" for _, s in a.made) and not a.recorded


def test_every_binding_with_a_stream_is_listed():
    import inspect
    takes = {n for n, f in vars(moeq).items()
             if n.startswith("moe_") and inspect.isfunction(f) and "stream" in inspect.signature(f).parameters}
    assert takes == set(CALLS)
