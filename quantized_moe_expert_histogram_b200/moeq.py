"""Thin ctypes binding of libmoeq.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does
nothing but check tensor dtypes/devices, pass raw pointers and sizes, and
turn a non-zero status into an exception.  All arithmetic runs in the CUDA
kernels of the library; there is no CPU fallback: ``load()`` raises when
the library is missing or no CUDA device is present.

``stream=`` (a ``torch.cuda.Stream``; the current one when left out) is where
a call's kernels run.  Outputs and workspaces that the call makes itself
belong to that stream, as if made under ``torch.cuda.stream(stream)``; a
caller who goes on with an output elsewhere makes that stream wait, as for
any tensor.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoeq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "moeq.h")

LAYOUT_INT4 = 0
LAYOUT_PLANES = 1
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
DEV_BAD_INDEX = 1
DEV_RANGE = 2
DEV_TIMEOUT = 4

_c_p = ctypes.c_void_p
_c_i = ctypes.c_int
_c_sz = ctypes.c_size_t

_SIGS = {
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_blob_bytes": (_c_sz, [_c_i, _c_i, _c_i, _c_i]),
    "moe_quant_pack": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p]),
    "moe_route_topk": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p, _c_sz,
                              _c_p]),
    "moe_route_workspace_bytes": (_c_sz, [_c_i, _c_i, _c_i]),
    "moe_route_topk_noalloc": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p]),
    "moe_route_scored": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i,
                                ctypes.c_double, _c_p, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "moe_route_scored_workspace_bytes": (_c_sz, [_c_i, _c_i, _c_i]),
    "moe_permute": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p, _c_p, _c_p,
                           _c_p, _c_p, _c_sz, _c_p]),
    "moe_permute_workspace_bytes": (_c_sz, [_c_i, _c_i, _c_i, _c_i]),
    "moe_route_permute": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p,
                                 _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "moe_route_permute_workspace_bytes": (_c_sz, [_c_i, _c_i, _c_i, _c_i, _c_i]),
    "moe_static_bits": (_c_i, [_c_p, _c_p, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p]),
    "moe_bit_gate": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p]),
    "moe_ffn_workspace_bytes": (_c_sz, [_c_i, _c_i, _c_i, _c_i, _c_i]),
    "moe_grouped_ffn_wq": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i,
                                  _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "moe_unpermute_combine": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_p, _c_p]),
    "moe_grouped_ffn_combine": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p,
                                       _c_p, _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "moe_ffn_combine_workspace_bytes": (_c_sz, [_c_i, _c_i, _c_i, _c_i, _c_i, _c_i]),
    "moe_mx_matrix_bytes": (_c_sz, [_c_i, _c_i]),
    "moe_mx_blob_bytes": (_c_sz, [_c_i, _c_i]),
    "moe_mx_quantize": (_c_i, [_c_p, _c_i, _c_i, _c_i, _c_sz, _c_p, _c_i, _c_p, _c_p, _c_p, _c_p]),
    "moe_mx_dequantize": (_c_i, [_c_p, _c_p, _c_i, _c_i, _c_i, _c_p, _c_p]),
    "moe_mx_pack": (_c_i, [_c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p]),
    "moe_mx_pack_ffn": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p]),
    "moe_mx_grouped_gemm": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p]),
    "moe_grouped_ffn_mx": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "moe_ffn_mx_workspace_bytes": (_c_sz, [_c_i, _c_i]),
    "moe_slot_cache_create": (_c_i, [_c_i, _c_i, _c_sz, _c_p, _c_p, ctypes.POINTER(_c_p)]),
    "moe_slot_cache_create_planes": (_c_i, [_c_i, _c_i, _c_i, _c_i, _c_i, _c_p, _c_p, ctypes.POINTER(_c_p)]),
    "moe_slot_stage": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_p, _c_p, _c_p, _c_p]),
    "moe_slot_ffn": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i, _c_i, _c_i, _c_i, _c_i, _c_p, _c_sz, _c_p,
                            _c_p, _c_p, _c_p]),
    "moe_slot_cache_destroy": (None, [_c_p]),
    "moe_slot_prefetch": (_c_i, [_c_p, _c_p, _c_i, _c_i, _c_p, _c_p]),
    "moe_slot_timing": (_c_i, [_c_p, _c_i]),
    "moe_slot_timing_read": (_c_i, [_c_p, _c_p, _c_p]),
    "moe_predictor_create": (_c_i, [_c_i, _c_i, ctypes.POINTER(_c_p)]),
    "moe_predictor_destroy": (None, [_c_p]),
    "moe_predictor_observe": (_c_i, [_c_p, _c_i, _c_p, _c_p, _c_p, _c_i, _c_i]),
    "moe_predictor_predict": (_c_i, [_c_p, _c_i, _c_p, _c_p, _c_i, _c_i, _c_i, ctypes.c_double, _c_p, _c_p]),
    "moe_debug_inject_fault": (None, [_c_i, _c_i]),
    "moe_debug_force_regime": (None, [_c_i]),
    "moe_debug_set_trace": (None, [_c_p]),
    "moe_debug_ffn_timeout": (None, [_c_i]),
    "moe_debug_mx_timeout": (None, [_c_i]),
    "moe_debug_route_fused": (None, [_c_i]),
}

_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


def header_symbols() -> list:
    """Names of the functions declared in include/moeq.h."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"MOE_API\s+[\w\s\*]+?\b(moe_\w+)\s*\(", text)


def open_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """dlopen the library and attach signatures (needs no GPU)."""
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run quantized_moe_expert_histogram_b200.build.build()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


def load():
    """The library, for compute calls; raises without a CUDA device."""
    global _lib
    if _lib is not None:
        return _lib
    if not torch.cuda.is_available():
        raise RuntimeError("moeq needs a CUDA device (B200, sm_100a); no CPU fallback exists")
    _lib = open_library()
    return _lib


def _check(fn, code):
    if code != 0:
        raise MoeError(fn, code, _lib.moe_last_error().decode())


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (3 us of a
# decode step's host time for every call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _new(like, shape, dtype, stream, scratch=False):
    """A new tensor on the device of `like` for a call on `stream`.

    Its memory comes from the pool of the stream that the call runs on: a
    block that another stream released may still be read by that stream's
    queued work.  The tensor returned belongs to that stream; the current
    stream, on which the caller goes on to use it (after waiting), is recorded
    as a user, so that the memory is not given out again before it has passed
    the tensor's release.  scratch: for this call only, dropped before it
    returns."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    current = torch.cuda.current_stream(like.device)
    if stream == current:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if not scratch:
        t.record_stream(current)
    return t


def _holds(fn, name, t, n):
    """t, if given, has the n elements that the call reads or writes."""
    if t is not None and t.numel() < n:
        raise ValueError(f"{fn}: {name} must hold {n} elements, got {tuple(t.shape)}")


def moe_blob_bytes(d, F, group, layout):
    return int(load().moe_blob_bytes(d, F, group, layout))


def moe_ffn_workspace_bytes(total_rows, E, d, F, layout):
    return int(load().moe_ffn_workspace_bytes(total_rows, E, d, F, layout))


def moe_quant_pack(w_gate, w_up, w_down, group, layout, blobs=None, stream=None):
    lib = load()
    E, F, d = w_gate.shape
    nb = lib.moe_blob_bytes(d, F, group, layout)
    if blobs is None:
        blobs = _new(w_gate, (E, nb), torch.uint8, stream)
    _check("moe_quant_pack", lib.moe_quant_pack(
        _ptr(w_gate, torch.float32, "w_gate"), _ptr(w_up, torch.float32, "w_up"),
        _ptr(w_down, torch.float32, "w_down"), E, d, F, group, layout,
        _ptr(blobs, torch.uint8, "blobs"), _stream(stream)))
    return blobs


def moe_route_workspace_bytes(T, d, E):
    return int(load().moe_route_workspace_bytes(T, d, E))


def moe_route_topk(x, w_router, bias, k, forced_idx=None, topk_idx=None, topk_w=None, workspace=None,
                   stream=None):
    lib = load()
    T, d = x.shape
    E = w_router.shape[0]
    if topk_idx is None:
        topk_idx = _new(x, (T, k), torch.int32, stream)
    if topk_w is None:
        topk_w = _new(x, (T, k), torch.float32, stream)
    if workspace is None:
        workspace = _new(x, (lib.moe_route_workspace_bytes(T, d, E),), torch.uint8, stream, scratch=True)
    _check("moe_route_topk", lib.moe_route_topk(
        _ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.float32, "w_router"),
        _ptr(bias, torch.float32, "bias"), _ptr(forced_idx, torch.int32, "forced_idx"), T, d, E, k,
        _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(topk_w, torch.float32, "topk_w"),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return topk_idx, topk_w


def moe_permute_workspace_bytes(T, E, k, nested):
    return int(load().moe_permute_workspace_bytes(T, E, k, int(bool(nested))))


def moe_permute(topk_idx, E, bits=None, x=None, out=None, status=None, workspace=None, stream=None):
    """Returns dict(counts, offsets, perm, inv_perm, x_perm)."""
    lib = load()
    T, k = topk_idx.shape
    nb = 3 * E if bits is not None else E
    d = x.shape[1] if x is not None else 0
    if out is None:
        out = dict(counts=_new(topk_idx, (nb,), torch.int32, stream),
                   offsets=_new(topk_idx, (nb + 1,), torch.int32, stream),
                   perm=_new(topk_idx, (T * k,), torch.int32, stream),
                   inv_perm=_new(topk_idx, (T * k,), torch.int32, stream),
                   x_perm=_new(topk_idx, (T * k, d), torch.float16, stream) if x is not None else None)
    if workspace is None:
        workspace = out.get("perm_ws")
    if workspace is None:
        workspace = _new(topk_idx, (lib.moe_permute_workspace_bytes(T, E, k, int(bits is not None)),), torch.uint8,
                         stream, scratch=True)
    _check("moe_permute", lib.moe_permute(
        _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(bits, torch.uint8, "bits"),
        _ptr(x, torch.bfloat16, "x"), T, d, E, k, _ptr(out["counts"], torch.int32),
        _ptr(out["offsets"], torch.int32), _ptr(out["perm"], torch.int32),
        _ptr(out["inv_perm"], torch.int32), _ptr(out["x_perm"], torch.float16),
        _ptr(status, torch.int32, "status"), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out


def moe_route_permute_workspace_bytes(T, d, E, k, nested):
    return int(load().moe_route_permute_workspace_bytes(T, d, E, k, int(bool(nested))))


def moe_route_permute(x, w_router, bias, k, forced_idx=None, bits=None, w_bit=None, bias_bit=None, out=None,
                      status=None, workspace=None, gather=True, stream=None):
    """Router, optional bit gate (w_bit) or given widths (bits), and the
    permutation in one call.  Returns dict(topk_idx, topk_w, bits, counts,
    offsets, perm, inv_perm, x_perm); 'bits' holds the gate's widths (or the
    given ones, or None)."""
    lib = load()
    T, d = x.shape
    E = w_router.shape[0]
    nested = bits is not None or w_bit is not None
    nb = 3 * E if nested else E
    if out is None:
        out = {}
    out = dict(out)
    for key, shape, dt in (("topk_idx", (T, k), torch.int32), ("topk_w", (T, k), torch.float32),
                           ("counts", (nb,), torch.int32), ("offsets", (nb + 1,), torch.int32),
                           ("perm", (T * k,), torch.int32), ("inv_perm", (T * k,), torch.int32)):
        if out.get(key) is None:
            out[key] = _new(x, shape, dt, stream)
    if gather and out.get("x_perm") is None:
        out["x_perm"] = _new(x, (T * k, d), torch.float16, stream)
    bits_out = None
    if w_bit is not None:
        bits_out = out.get("bits")
        if bits_out is None:
            bits_out = _new(x, (T, k), torch.uint8, stream)
    if workspace is None:
        workspace = _new(x, (lib.moe_route_permute_workspace_bytes(T, d, E, k, int(nested)),), torch.uint8, stream,
                         scratch=True)
    _check("moe_route_permute", lib.moe_route_permute(
        _ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.float32, "w_router"), _ptr(bias, torch.float32, "bias"),
        _ptr(forced_idx, torch.int32, "forced_idx"), _ptr(bits, torch.uint8, "bits"),
        _ptr(w_bit, torch.float32, "w_bit"), _ptr(bias_bit, torch.float32, "bias_bit"), T, d, E, k,
        _ptr(out["topk_idx"], torch.int32), _ptr(out["topk_w"], torch.float32), _ptr(bits_out, torch.uint8),
        _ptr(out["counts"], torch.int32), _ptr(out["offsets"], torch.int32), _ptr(out["perm"], torch.int32),
        _ptr(out["inv_perm"], torch.int32), _ptr(out["x_perm"] if gather else None, torch.float16),
        _ptr(status, torch.int32, "status"), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    out["bits"] = bits_out if w_bit is not None else bits
    return out


def moe_static_bits(topk_idx, width_of, E, bits=None, status=None, stream=None):
    """bits[t][j] = width_of[topk_idx[t][j]] (uint8 [T][k])."""
    lib = load()
    T, k = topk_idx.shape
    if bits is None:
        bits = _new(topk_idx, (T, k), torch.uint8, stream)
    _check("moe_static_bits", lib.moe_static_bits(
        _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(width_of, torch.uint8, "width_of"), T, k, E,
        _ptr(bits, torch.uint8, "bits"), _ptr(status, torch.int32, "status"), _stream(stream)))
    return bits


def moe_bit_gate(x, w_bit, bias_bit, topk_idx, bits=None, status=None, stream=None):
    """bits[t][j] = 2 + argmax_c (x[t] . w_bit[e][c] + bias_bit[e][c]) for
    e = topk_idx[t][j] (uint8 [T][k])."""
    lib = load()
    T, d = x.shape
    E = w_bit.shape[0]
    k = topk_idx.shape[1]
    if bits is None:
        bits = _new(x, (T, k), torch.uint8, stream)
    _check("moe_bit_gate", lib.moe_bit_gate(
        _ptr(x, torch.bfloat16, "x"), _ptr(w_bit, torch.float32, "w_bit"),
        _ptr(bias_bit, torch.float32, "bias_bit"), _ptr(topk_idx, torch.int32, "topk_idx"), T, d, E, k,
        _ptr(bits, torch.uint8, "bits"), _ptr(status, torch.int32, "status"), _stream(stream)))
    return bits


def moe_ffn_combine_workspace_bytes(T, k, E, d, F, layout):
    return int(load().moe_ffn_combine_workspace_bytes(T, k, E, d, F, layout))


def moe_grouped_ffn_combine(x_perm, offsets, blobs, T, k, E, d, F, group, layout, perm, inv_perm, topk_w,
                            residual=None, y=None, y_perm=None, workspace=None, status=None, stream=None):
    """The grouped FFN and the weighted combine in one call; returns (y, y_perm)."""
    lib = load()
    _holds("moe_grouped_ffn_combine", "residual", residual, T * d)
    _holds("moe_grouped_ffn_combine", "y", y, T * d)
    if y is None:
        y = _new(x_perm, (T, d), torch.bfloat16, stream)
    if y_perm is None:
        y_perm = _new(x_perm, (T * k, d), torch.float16, stream)
    if workspace is None:
        workspace = _new(x_perm, (lib.moe_ffn_combine_workspace_bytes(T, k, E, d, F, layout),), torch.uint8, stream,
                         scratch=True)
    _check("moe_grouped_ffn_combine", lib.moe_grouped_ffn_combine(
        _ptr(x_perm, torch.float16, "x_perm"), _ptr(offsets, torch.int32, "offsets"), _ptr(blobs), T, k, E, d, F,
        group, layout, _ptr(perm, torch.int32, "perm"), _ptr(inv_perm, torch.int32, "inv_perm"),
        _ptr(topk_w, torch.float32, "topk_w"), _ptr(residual, torch.bfloat16, "residual"),
        _ptr(y, torch.bfloat16, "y"), _ptr(y_perm, torch.float16, "y_perm"), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(status, torch.int32, "status"), _stream(stream)))
    return y, y_perm


def moe_grouped_ffn_wq(x_perm, offsets, blobs, T, E, d, F, group, layout, slot_of=None,
                       workspace=None, y_perm=None, status=None, stream=None):
    lib = load()
    rows = x_perm.shape[0]
    if workspace is None:
        workspace = _new(x_perm, (lib.moe_ffn_workspace_bytes(rows, E, d, F, layout),), torch.uint8, stream,
                         scratch=True)
    if y_perm is None:
        y_perm = _new(x_perm, (rows, d), torch.float16, stream)
    _check("moe_grouped_ffn_wq", lib.moe_grouped_ffn_wq(
        _ptr(x_perm, torch.float16, "x_perm"), _ptr(offsets, torch.int32, "offsets"), _ptr(blobs),
        _ptr(slot_of, torch.int32, "slot_of"), rows, T, E, d, F, group, layout, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(y_perm, torch.float16, "y_perm"),
        _ptr(status, torch.int32, "status"), _stream(stream)))
    return y_perm


def moe_unpermute_combine(y_perm, inv_perm, topk_w, residual=None, y=None, stream=None):
    lib = load()
    T, k = topk_w.shape
    d = y_perm.shape[1]
    for name, t, n in (("y_perm", y_perm, T * k * d), ("inv_perm", inv_perm, T * k), ("residual", residual, T * d),
                       ("y", y, T * d)):
        _holds("moe_unpermute_combine", name, t, n)
    if y is None:
        y = _new(y_perm, (T, d), torch.bfloat16, stream)
    _check("moe_unpermute_combine", lib.moe_unpermute_combine(
        _ptr(y_perm, torch.float16, "y_perm"), _ptr(inv_perm, torch.int32, "inv_perm"),
        _ptr(topk_w, torch.float32, "topk_w"), _ptr(residual, torch.bfloat16, "residual"), T, k, d,
        _ptr(y, torch.bfloat16, "y"), _stream(stream)))
    return y


# ---- scored router and MXFP4 ------------------------------------------------
#
# A decode step's calls are bound by the host, so the checks here are few and
# cheap (the sizes that only the library knows are checked there).

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_SCORING = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


class _Other:
    """Runs a call with another device current (a call's launches belong to
    the current one)."""

    __slots__ = ("guard",)

    def __init__(self, device):
        self.guard = torch.cuda.device(device)

    def __enter__(self):
        self.guard.__enter__()

    def __exit__(self, *exc):
        self.guard.__exit__(*exc)


class _Same:
    __slots__ = ()

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_SAME = _Same()


def _on(fn, first, *others):
    """A context in which the tensors' own device is current; tensors on
    different devices are refused."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError(f"{fn}: the tensors must be on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{fn}: tensors on {first.device} and {t.device}")
    return _SAME if dev == torch.cuda.current_device() else _Other(dev)


def _sized(fn, name, t, shape):
    if t is not None and t.shape != shape:
        raise ValueError(f"{fn}: {name} must have shape {shape}, got {tuple(t.shape)}")


def _dtype_id(fn, name, dtype):
    if dtype not in _DTYPE:
        raise TypeError(f"{fn}: {name} must be float32, bfloat16 or float16, got {dtype}")
    return _DTYPE[dtype]


def moe_route_scored_workspace_bytes(T, d, E):
    return int(load().moe_route_scored_workspace_bytes(T, d, E))


def moe_route_scored(x, w_router, k, scoring="softmax", bias=None, n_groups=1, topk_groups=1, group_top=1,
                     renorm=True, scale=1.0, topk_idx=None, topk_w=None, workspace=None, status=None, stream=None):
    """Router with softmax or sigmoid scores, a balance bias, expert groups
    and renormalised weights; returns (topk_idx, topk_w)."""
    lib = load()
    fn = "moe_route_scored"
    if scoring not in _SCORING:
        raise ValueError(f"{fn}: scoring must be 'softmax' or 'sigmoid', got {scoring!r}")
    T, d = x.shape
    E = w_router.shape[0]
    _sized(fn, "w_router", w_router, (E, d))
    _sized(fn, "bias", bias, (E,))
    _sized(fn, "topk_idx", topk_idx, (T, k))
    _sized(fn, "topk_w", topk_w, (T, k))
    with _on(fn, x, w_router, bias, topk_idx, topk_w, workspace, status):
        if topk_idx is None:
            topk_idx = _new(x, (T, k), torch.int32, stream)
        if topk_w is None:
            topk_w = _new(x, (T, k), torch.float32, stream)
        if workspace is None:
            workspace = _new(x, (lib.moe_route_scored_workspace_bytes(T, d, E),), torch.uint8, stream, scratch=True)
        _check(fn, lib.moe_route_scored(
            _ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.float32, "w_router"), _ptr(bias, torch.float32, "bias"),
            T, d, E, k, _SCORING[scoring], n_groups, topk_groups, group_top, 1 if renorm else 0, scale,
            _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(topk_w, torch.float32, "topk_w"), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(status, torch.int32, "status"), _stream(stream)))
    return topk_idx, topk_w


def moe_mx_matrix_bytes(N, K):
    return int(load().moe_mx_matrix_bytes(N, K))


def moe_mx_blob_bytes(d, F):
    return int(load().moe_mx_blob_bytes(d, F))


def moe_mx_quantize(x, inv_perm=None, k=1, codes=None, scales=None, status=None, stream=None):
    """Rows of x (fp32, bf16 or fp16; rows may be strided) to MXFP4; with
    inv_perm (from moe_permute) row t goes to its k places.  Returns (codes
    uint8 [rows * k][K/2], scales uint8 [rows * k][K/32])."""
    lib = load()
    fn = "moe_mx_quantize"
    rows, K = x.shape
    ld, step = x.stride()
    dt = _dtype_id(fn, "x", x.dtype)
    if rows <= 1:
        ld = K
    if (K > 1 and step != 1) or ld < K:
        raise ValueError(f"{fn}: x must have contiguous rows that do not overlap")
    if inv_perm is not None and inv_perm.numel() != rows * k:
        raise ValueError(f"{fn}: inv_perm must hold rows * k = {rows * k} places, got {inv_perm.numel()}")
    _sized(fn, "codes", codes, (rows * k, K // 2))
    _sized(fn, "scales", scales, (rows * k, K // 32))
    with _on(fn, x, inv_perm, codes, scales, status):
        if codes is None:
            codes = _new(x, (rows * k, K // 2), torch.uint8, stream)
        if scales is None:
            scales = _new(x, (rows * k, K // 32), torch.uint8, stream)
        _check(fn, lib.moe_mx_quantize(
            x.data_ptr(), dt, rows, K, ld, _ptr(inv_perm, torch.int32, "inv_perm"), k,
            _ptr(codes, torch.uint8, "codes"), _ptr(scales, torch.uint8, "scales"),
            _ptr(status, torch.int32, "status"), _stream(stream)))
    return codes, scales


def moe_mx_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values of MXFP4 rows, [rows][K] in bf16 or fp32 (exact)."""
    lib = load()
    fn = "moe_mx_dequantize"
    rows, K = codes.shape
    K *= 2
    dt = _dtype_id(fn, "dtype", dtype)
    _sized(fn, "scales", scales, (rows, K // 32))
    _sized(fn, "out", out, (rows, K))
    with _on(fn, codes, scales, out):
        if out is None:
            out = _new(codes, (rows, K), dtype, stream)
        _check(fn, lib.moe_mx_dequantize(_ptr(codes, torch.uint8, "codes"), _ptr(scales, torch.uint8, "scales"), rows,
                                         K, dt, _ptr(out, dtype, "out"), _stream(stream)))
    return out


def moe_mx_pack(w, mats=None, status=None, stream=None):
    """Matrices w [E][N][K] (fp32, bf16 or fp16) to MXFP4, uint8 [E][bytes]."""
    lib = load()
    fn = "moe_mx_pack"
    E, N, K = w.shape
    dt = _dtype_id(fn, "w", w.dtype)
    nb = lib.moe_mx_matrix_bytes(N, K)
    _sized(fn, "mats", mats, (E, nb))
    with _on(fn, w, mats, status):
        if mats is None:
            mats = _new(w, (E, nb), torch.uint8, stream)
        _check(fn, lib.moe_mx_pack(_ptr(w, None, "w"), dt, E, N, K, _ptr(mats, torch.uint8, "mats") or None,
                                   _ptr(status, torch.int32, "status"), _stream(stream)))
    return mats


def moe_mx_pack_ffn(w_gate, w_up, w_down, blobs=None, status=None, stream=None):
    """w_gate, w_up [E][F][d] and w_down [E][d][F] (one dtype) to FFN blobs, uint8 [E][bytes]."""
    lib = load()
    fn = "moe_mx_pack_ffn"
    E, F, d = w_gate.shape
    dt = _dtype_id(fn, "w_gate", w_gate.dtype)
    _sized(fn, "w_up", w_up, (E, F, d))
    _sized(fn, "w_down", w_down, (E, d, F))
    nb = lib.moe_mx_blob_bytes(d, F)
    _sized(fn, "blobs", blobs, (E, nb))
    with _on(fn, w_gate, w_up, w_down, blobs, status):
        if blobs is None:
            blobs = _new(w_gate, (E, nb), torch.uint8, stream)
        _check(fn, lib.moe_mx_pack_ffn(
            _ptr(w_gate, None, "w_gate"), _ptr(w_up, w_gate.dtype, "w_up"), _ptr(w_down, w_gate.dtype, "w_down"), dt,
            E, d, F, _ptr(blobs, torch.uint8, "blobs") or None, _ptr(status, torch.int32, "status"), _stream(stream)))
    return blobs


def _mx_args(fn, codes, scales, offsets, mats, nbytes):
    rows, K = codes.shape
    K *= 2
    E = mats.shape[0]
    _sized(fn, "scales", scales, (rows, K // 32))
    _sized(fn, "offsets", offsets, (E + 1,))
    if nbytes and mats.numel() != E * nbytes:
        raise ValueError(f"{fn}: the weights must hold {nbytes} bytes per expert, got {mats.numel() // max(E, 1)}")
    return rows, K, E


def moe_mx_grouped_gemm(codes, scales, offsets, mats, N, dtype=torch.float16, out=None, status=None, stream=None):
    """y[p] = W_e xq[p] for the rows of each expert; returns [rows][N] in dtype."""
    lib = load()
    fn = "moe_mx_grouped_gemm"
    dt = _dtype_id(fn, "dtype", dtype)
    rows, K, E = _mx_args(fn, codes, scales, offsets, mats, lib.moe_mx_matrix_bytes(N, codes.shape[1] * 2))
    _sized(fn, "out", out, (rows, N))
    with _on(fn, codes, scales, offsets, mats, out, status):
        if out is None:
            out = _new(codes, (rows, N), dtype, stream)
        _check(fn, lib.moe_mx_grouped_gemm(
            _ptr(codes, torch.uint8, "codes"), _ptr(scales, torch.uint8, "scales"),
            _ptr(offsets, torch.int32, "offsets"), _ptr(mats, torch.uint8, "mats"), rows, E, N, K, dt,
            _ptr(out, dtype, "out"), _ptr(status, torch.int32, "status"), _stream(stream)))
    return out


def moe_ffn_mx_workspace_bytes(rows, F):
    return int(load().moe_ffn_mx_workspace_bytes(rows, F))


def moe_grouped_ffn_mx(codes, scales, offsets, blobs, F, workspace=None, y_perm=None, status=None, stream=None):
    """The grouped expert FFN on MXFP4 rows and blobs; returns y_perm fp16 [rows][d]."""
    lib = load()
    fn = "moe_grouped_ffn_mx"
    rows, d, E = _mx_args(fn, codes, scales, offsets, blobs, lib.moe_mx_blob_bytes(codes.shape[1] * 2, F))
    _sized(fn, "y_perm", y_perm, (rows, d))
    with _on(fn, codes, scales, offsets, blobs, workspace, y_perm, status):
        if workspace is None:
            workspace = _new(codes, (lib.moe_ffn_mx_workspace_bytes(rows, F),), torch.uint8, stream, scratch=True)
        if y_perm is None:
            y_perm = _new(codes, (rows, d), torch.float16, stream)
        _check(fn, lib.moe_grouped_ffn_mx(
            _ptr(codes, torch.uint8, "codes"), _ptr(scales, torch.uint8, "scales"),
            _ptr(offsets, torch.int32, "offsets"), _ptr(blobs, torch.uint8, "blobs"), rows, E, d, F, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(y_perm, torch.float16, "y_perm"),
            _ptr(status, torch.int32, "status"), _stream(stream)))
    return y_perm


class SlotCache:
    """One layer's GPU slot cache (moe_slot_cache_create / _destroy); with
    planes=(d, F, group) a plane-mode cache of nested-plane blobs
    (moe_slot_cache_create_planes)."""

    def __init__(self, E, slots, blob_bytes, host_blobs, device_pool, planes=None):
        lib = load()
        if not host_blobs.is_pinned():
            raise ValueError("host_blobs must be pinned host memory")
        self._host = host_blobs
        self._pool = device_pool
        h = _c_p()
        if planes is None:
            _check("moe_slot_cache_create", lib.moe_slot_cache_create(
                E, slots, blob_bytes, host_blobs.data_ptr(), _ptr(device_pool), ctypes.byref(h)))
        else:
            d, F, group = planes
            moe_slot_cache_create_planes(E, slots, d, F, group, host_blobs, device_pool, h)
        self.handle = h
        self.E = E
        self._ids = None

    def stage(self, ids_host, copy_stream, compute_stream, bits_host=None):
        """moe_slot_stage; returns (n_waves, [hits, experts copied, bytes])."""
        lib = load()
        ids = ids_host.to(torch.int32).contiguous()
        bits = None if bits_host is None else bits_host.to(torch.uint8).contiguous().cpu()
        self._ids, self._bits = ids, bits
        nw = ctypes.c_int32(0)
        stats = (ctypes.c_int64 * 3)()
        _check("moe_slot_stage", lib.moe_slot_stage(
            self.handle, ids.data_ptr(), None if bits is None else bits.data_ptr(), ids.numel(),
            copy_stream.cuda_stream, compute_stream.cuda_stream, ctypes.byref(nw), stats))
        return nw.value, list(stats)

    def ffn(self, x_perm, offsets, T, d, F, group, layout, workspace, y_perm, status, copy_stream,
            compute_stream):
        lib = load()
        _check("moe_slot_ffn", lib.moe_slot_ffn(
            self.handle, _ptr(x_perm, torch.float16), _ptr(offsets, torch.int32), x_perm.shape[0], T,
            d, F, group, layout, _ptr(workspace), workspace.numel() * workspace.element_size(),
            _ptr(y_perm, torch.float16), _ptr(status, torch.int32), copy_stream.cuda_stream,
            compute_stream.cuda_stream))

    def prefetch(self, ids_host, max_copies, copy_stream):
        """moe_slot_prefetch: stage up to max_copies of the listed experts
        ahead of their layer-step; returns the number of copies issued."""
        return moe_slot_prefetch(self.handle, ids_host, max_copies, copy_stream)

    def timing(self, enable):
        """moe_slot_timing: record copy and FFN busy time from now on."""
        moe_slot_timing(self.handle, enable)

    def timing_read(self):
        """moe_slot_timing_read: (copy_ms, ffn_ms) since the last read."""
        return moe_slot_timing_read(self.handle)

    def close(self):
        if self.handle is not None and self.handle.value:
            load().moe_slot_cache_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_slot_prefetch(handle, ids_host, max_copies, copy_stream):
    ids = ids_host.to(torch.int32).contiguous()
    n = ctypes.c_int32(0)
    _check("moe_slot_prefetch", load().moe_slot_prefetch(handle, ids.data_ptr(), ids.numel(), int(max_copies),
                                                          copy_stream.cuda_stream, ctypes.byref(n)))
    return n.value


def moe_slot_cache_create_planes(E, slots, d, F, group, host_blobs, device_pool, handle):
    _check("moe_slot_cache_create_planes", load().moe_slot_cache_create_planes(
        E, slots, d, F, group, host_blobs.data_ptr(), _ptr(device_pool), ctypes.byref(handle)))
    return handle


def moe_slot_timing(handle, enable):
    _check("moe_slot_timing", load().moe_slot_timing(handle, int(bool(enable))))


def moe_slot_timing_read(handle):
    cm, fm = ctypes.c_double(0), ctypes.c_double(0)
    _check("moe_slot_timing_read", load().moe_slot_timing_read(handle, ctypes.addressof(cm), ctypes.addressof(fm)))
    return cm.value, fm.value


def moe_predictor_create(layers, E):
    h = _c_p()
    _check("moe_predictor_create", load().moe_predictor_create(layers, E, ctypes.byref(h)))
    return h


def moe_predictor_destroy(handle):
    load().moe_predictor_destroy(handle)


def _host_ids(ids):
    return None if ids is None else ids.to(torch.int32).contiguous().cpu()


def moe_predictor_observe(handle, layer, prev_ids, cur_ids, prev2_ids=None):
    prev, cur, prev2 = _host_ids(prev_ids), _host_ids(cur_ids), _host_ids(prev2_ids)
    T, k = prev.shape
    _check("moe_predictor_observe", load().moe_predictor_observe(
        handle, layer, None if prev2 is None else prev2.data_ptr(), prev.data_ptr(), cur.data_ptr(), T, k))


def moe_predictor_predict(handle, layer, prev_ids, max_out, min_score=0.0, prev2_ids=None):
    prev, prev2 = _host_ids(prev_ids), _host_ids(prev2_ids)
    T, k = prev.shape
    out = torch.empty(max(1, max_out), dtype=torch.int32)
    n = ctypes.c_int32(0)
    _check("moe_predictor_predict", load().moe_predictor_predict(
        handle, layer, None if prev2 is None else prev2.data_ptr(), prev.data_ptr(), T, k, max_out,
        float(min_score), out.data_ptr(), ctypes.byref(n)))
    return out[:n.value]


class RoutePredictor:
    """Next-layer expert predictor (moe_predictor_*), host-side."""

    def __init__(self, layers, E):
        self.handle = moe_predictor_create(layers, E)

    def observe(self, layer, prev_ids, cur_ids, prev2_ids=None):
        moe_predictor_observe(self.handle, layer, prev_ids, cur_ids, prev2_ids)

    def predict(self, layer, prev_ids, max_out, min_score=0.0, prev2_ids=None):
        return moe_predictor_predict(self.handle, layer, prev_ids, max_out, min_score, prev2_ids)

    def close(self):
        if self.handle is not None and self.handle.value:
            moe_predictor_destroy(self.handle)
        self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_debug_inject_fault(what, count):
    load().moe_debug_inject_fault(what, count)


def moe_last_error():
    return load().moe_last_error().decode()


def moe_debug_force_regime(regime):
    """0 = by T, 1 = one-token GEMV, 2 = tensor cores, 3 = small-batch mma.sync kernel (test hook)."""
    load().moe_debug_force_regime(regime)


def moe_debug_route_fused(mode):
    """Test hook: 1 (default) one cluster launch for the smallest batches of
    the router, the bit gate and moe_route_permute; 0 the two-launch router,
    the one-kernel bit gate and separate launches at every size (see
    moeq.h)."""
    load().moe_debug_route_fused(int(mode))


def moe_debug_ffn_timeout(enable):
    """Test hook: a withheld arrive and a 20 ms wait limit in the tensor-core FFN."""
    load().moe_debug_ffn_timeout(int(bool(enable)))


def moe_debug_mx_timeout(enable):
    """Test hook: the same in the MXFP4 product and the scored router's tensor-core logits."""
    load().moe_debug_mx_timeout(int(bool(enable)))


def moe_debug_set_trace(pinned_int32=None):
    """Progress record of the tensor-core FFN kernels (test hook)."""
    load().moe_debug_set_trace(None if pinned_int32 is None else pinned_int32.data_ptr())



def moe_route_topk_noalloc(x, w_router, bias, k, forced_idx=None, topk_idx=None, topk_w=None, stream=None):
    """The router without a workspace argument: its scratch is a fixed
    device array inside the library (see include/moeq.h)."""
    lib = load()
    T, d = x.shape
    E = w_router.shape[0]
    if topk_idx is None:
        topk_idx = _new(x, (T, k), torch.int32, stream)
    if topk_w is None:
        topk_w = _new(x, (T, k), torch.float32, stream)
    _check("moe_route_topk_noalloc", lib.moe_route_topk_noalloc(
        _ptr(x, torch.bfloat16, "x"), _ptr(w_router, torch.float32, "w_router"),
        _ptr(bias, torch.float32, "bias"), _ptr(forced_idx, torch.int32, "forced_idx"), T, d, E, k,
        _ptr(topk_idx, torch.int32, "topk_idx"), _ptr(topk_w, torch.float32, "topk_w"), _stream(stream)))
    return topk_idx, topk_w
