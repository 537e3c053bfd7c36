"""Python binding of the MI355X MoE FFN layer library (libcolibri_moe.so).

Argument marshalling only: the functions below carry the C ABI's names
(``include/colibri_moe.h``) and pass plain pointers and sizes through ctypes;
every step of the layer runs in the library's HIP kernels. PyTorch is used for
device memory and streams only (``MoELayer``). There is no CPU fallback: if the
library is missing or fails to load, importing the layer raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcolibri_moe.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_OUT_OF_MEMORY, ERR_HIP, ERR_TOO_LARGE = range(7)
STATIC_SCRATCH_BYTES = 64 << 20  # COLIBRI_MOE_STATIC_SCRATCH_BYTES
FEW_TOKENS = 16  # COLIBRI_MOE_FEW_TOKENS
INT4_ROWS = 128  # COLIBRI_MOE_INT4_ROWS
F32, BF16, F16 = 0, 1, 2
FLAG_ASYNC = 1 << 0
FLAG_STAGE_TIMING = 1 << 1
FLAG_FP8_WEIGHTS = 1 << 2
FLAG_FP8_ACTIVATIONS = 1 << 3
FLAG_MXFP4_WEIGHTS = 1 << 4
FLAG_MXFP4_ACTIVATIONS = 1 << 5
STAGES = ("router", "dispatch", "gate_up_gemm", "gate_up_reduce", "down_gemm", "combine")


class Config(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class Weights(ctypes.Structure):
    _fields_ = [("w_router", ctypes.c_void_p), ("b_router", ctypes.c_void_p), ("w_gate", ctypes.c_void_p),
                ("w_up", ctypes.c_void_p), ("w_down", ctypes.c_void_p)]


class Routing(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("topk_ids", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
                ("expert_counts", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("perm_slot", ctypes.c_void_p), ("inv", ctypes.c_void_p)]


class Rule(ctypes.Structure):
    _fields_ = [("scoring", ctypes.c_int), ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int), ("normalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class Norm(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_stride", ctypes.c_int64), ("residual", ctypes.c_void_p),
                ("residual_stride", ctypes.c_int64), ("weight", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("weight_dtype", ctypes.c_int), ("rows", ctypes.c_int64), ("cols", ctypes.c_int32),
                ("eps", ctypes.c_float), ("y", ctypes.c_void_p), ("residual_out", ctypes.c_void_p),
                ("residual_out_stride", ctypes.c_int64), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class Int4(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("group", ctypes.c_int32), ("scale_dtype", ctypes.c_int), ("swiglu", ctypes.c_int32)]


EXPORTS = ("colibri_moe_init", "colibri_moe_init_rule", "colibri_moe_forward", "colibri_moe_forward_static",
           "colibri_moe_forward_few", "colibri_moe_free",
           "colibri_moe_status_string", "colibri_moe_stage_times", "colibri_moe_stage_name",
           "colibri_moe_quantize_fp8", "colibri_moe_quantize_mxfp4", "colibri_moe_dequantize_mxfp4",
           "colibri_moe_route", "colibri_moe_rms_norm", "colibri_moe_quantize_int4", "colibri_moe_dequantize_int4",
           "colibri_moe_int4_bytes", "colibri_moe_int4_pack", "colibri_moe_int4_linear", "colibri_moe_stream_copy")

_lib = None


def lib() -> ctypes.CDLL:
    """Load libcolibri_moe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, i32 = ctypes.c_void_p, ctypes.c_int32
        L.colibri_moe_init.restype = ctypes.c_int
        L.colibri_moe_init.argtypes = [ctypes.POINTER(P), ctypes.POINTER(Config), ctypes.POINTER(Weights), P]
        L.colibri_moe_init_rule.restype = ctypes.c_int
        L.colibri_moe_init_rule.argtypes = [ctypes.POINTER(P), ctypes.POINTER(Config), ctypes.POINTER(Weights),
                                            ctypes.POINTER(Rule), P, P]
        L.colibri_moe_forward.restype = ctypes.c_int
        L.colibri_moe_forward.argtypes = [P, P, i32, P, ctypes.POINTER(Routing)]
        L.colibri_moe_forward_static.restype = ctypes.c_int
        L.colibri_moe_forward_static.argtypes = [P, P, i32, P, ctypes.POINTER(Routing)]
        L.colibri_moe_forward_few.restype = ctypes.c_int
        L.colibri_moe_forward_few.argtypes = [P, P, i32, P, ctypes.POINTER(Routing)]
        L.colibri_moe_free.restype = ctypes.c_int
        L.colibri_moe_free.argtypes = [P]
        L.colibri_moe_status_string.restype = ctypes.c_char_p
        L.colibri_moe_status_string.argtypes = [ctypes.c_int]
        L.colibri_moe_stage_times.restype = i32
        L.colibri_moe_stage_times.argtypes = [P, ctypes.POINTER(ctypes.c_float), i32]
        L.colibri_moe_stage_name.restype = ctypes.c_char_p
        L.colibri_moe_stage_name.argtypes = [i32]
        L.colibri_moe_quantize_fp8.restype = ctypes.c_int
        L.colibri_moe_quantize_fp8.argtypes = [P, ctypes.c_int64, ctypes.c_int64, P, P, P]
        L.colibri_moe_quantize_mxfp4.restype = ctypes.c_int
        L.colibri_moe_quantize_mxfp4.argtypes = [P, ctypes.c_int, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, P, P,
                                                 P]
        L.colibri_moe_dequantize_mxfp4.restype = ctypes.c_int
        L.colibri_moe_dequantize_mxfp4.argtypes = [P, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, P, P]
        L.colibri_moe_route.restype = ctypes.c_int
        L.colibri_moe_route.argtypes = [P, ctypes.c_int, ctypes.c_int64, i32, i32, i32, ctypes.POINTER(Rule), P, P, P, P]
        L.colibri_moe_rms_norm.restype = ctypes.c_int
        L.colibri_moe_rms_norm.argtypes = [ctypes.POINTER(Norm), P]
        i64, I4 = ctypes.c_int64, ctypes.POINTER(Int4)
        L.colibri_moe_quantize_int4.restype = ctypes.c_int
        L.colibri_moe_quantize_int4.argtypes = [P, ctypes.c_int, i64, i64, i64, i32, P, P, P, P]
        L.colibri_moe_dequantize_int4.restype = ctypes.c_int
        L.colibri_moe_dequantize_int4.argtypes = [P, P, ctypes.c_int, P, i64, i64, i32, ctypes.c_int, P, P]
        L.colibri_moe_int4_bytes.restype = i64
        L.colibri_moe_int4_bytes.argtypes = [I4]
        L.colibri_moe_int4_pack.restype = ctypes.c_int
        L.colibri_moe_int4_pack.argtypes = [I4, P, P, P, P, P]
        L.colibri_moe_int4_linear.restype = ctypes.c_int
        L.colibri_moe_int4_linear.argtypes = [I4, P, P, i32, i32, i32, P, P, P, ctypes.c_int, P]
        L.colibri_moe_stream_copy.restype = ctypes.c_int
        L.colibri_moe_stream_copy.argtypes = [P, P, ctypes.c_int64, P]
        _lib = L
    return _lib


# --- the C ABI, one Python function per entry point -------------------------

def colibri_moe_init(cfg: Config, weights: Weights, hip_stream: int = 0):
    """Returns (status, handle)."""
    h = ctypes.c_void_p()
    st = lib().colibri_moe_init(ctypes.byref(h), ctypes.byref(cfg), ctypes.byref(weights),
                                ctypes.c_void_p(hip_stream))
    return st, h.value


def colibri_moe_init_rule(cfg: Config, weights: Weights, rule: Rule, bias_ptr, hip_stream: int = 0):
    """Returns (status, handle)."""
    h = ctypes.c_void_p()
    st = lib().colibri_moe_init_rule(ctypes.byref(h), ctypes.byref(cfg), ctypes.byref(weights),
                                     None if rule is None else ctypes.byref(rule), bias_ptr, hip_stream)
    return st, h.value


def colibri_moe_forward(handle, x_ptr: int, T: int, y_ptr: int, routing: Routing | None = None) -> int:
    return lib().colibri_moe_forward(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T, ctypes.c_void_p(y_ptr),
                                     None if routing is None else ctypes.byref(routing))


def colibri_moe_forward_static(handle, x_ptr: int, T: int, y_ptr: int, routing: Routing | None = None) -> int:
    return lib().colibri_moe_forward_static(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T,
                                            ctypes.c_void_p(y_ptr),
                                            None if routing is None else ctypes.byref(routing))


def colibri_moe_forward_few(handle, x_ptr: int, T: int, y_ptr: int, routing: Routing | None = None) -> int:
    return lib().colibri_moe_forward_few(ctypes.c_void_p(handle), ctypes.c_void_p(x_ptr), T, ctypes.c_void_p(y_ptr),
                                         None if routing is None else ctypes.byref(routing))


def colibri_moe_free(handle) -> int:
    return lib().colibri_moe_free(ctypes.c_void_p(handle))


def colibri_moe_status_string(status: int) -> str:
    return lib().colibri_moe_status_string(status).decode()


def colibri_moe_stage_times(handle) -> list:
    buf = (ctypes.c_float * len(STAGES))()
    n = lib().colibri_moe_stage_times(ctypes.c_void_p(handle), buf, len(STAGES))
    if n < 0:
        raise RuntimeError("stage timing not available (handle created without FLAG_STAGE_TIMING?)")
    return [float(buf[i]) for i in range(n)]


def colibri_moe_stage_name(stage: int):
    s = lib().colibri_moe_stage_name(stage)
    return None if s is None else s.decode()


def colibri_moe_quantize_fp8(w_ptr: int, rows: int, cols: int, codes_ptr: int, scales_ptr: int,
                             hip_stream: int = 0) -> int:
    return lib().colibri_moe_quantize_fp8(ctypes.c_void_p(w_ptr), rows, cols, ctypes.c_void_p(codes_ptr),
                                          ctypes.c_void_p(scales_ptr), ctypes.c_void_p(hip_stream))


def _stream_of(t, stream):
    """Handle of `stream`, or of the current stream of t's device (its raw
    handle: building a Stream object costs as much as the launch)."""
    import torch

    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(t.device.index)


def _on_device_of(t, fn, *args):
    """fn(*args) with t's device current (kernels run on the current one)."""
    import torch

    if t.device.index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(t.device):
        return fn(*args)


def _check_stream(stream, device):
    if stream.device != device:
        raise ValueError("the stream belongs to another device than the tensor")


def _empty_on(stream, device):
    """torch.empty for the outputs of a call on a given stream of `device`. Their
    memory is of that stream's own pool: what the allocator hands out of the
    current stream's pool may still be in use by kernels queued there, which
    nothing orders before `stream`. The current stream is recorded as a user,
    since the caller goes on there."""
    import torch

    _check_stream(stream, device)

    def empty(shape, dtype):
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
        t.record_stream(torch.cuda.current_stream(device))
        return t

    return empty


_I32_MAX = (1 << 31) - 1  # ctypes would cut a larger size, and the library answer for another one


def quantize_fp8(w, stream=None):
    """(codes uint8 [rows][cols], scales fp32 [rows]) of a contiguous bf16
    device tensor [rows][cols]: the 8-bit codes a layer built with
    FLAG_FP8_WEIGHTS keeps. Runs on `stream`, by default the current one, and
    waits for it; a given stream must already be ordered behind the work that
    makes w."""
    import torch

    if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_cuda or not w.is_contiguous():
        raise TypeError("w must be a contiguous 2-D bfloat16 device tensor")
    rows, cols = w.shape
    if stream is None:
        codes = torch.empty((rows, cols), dtype=torch.uint8, device=w.device)
        scales = torch.empty((rows,), dtype=torch.float32, device=w.device)
    else:
        empty = _empty_on(stream, w.device)
        codes, scales = empty((rows, cols), torch.uint8), empty((rows,), torch.float32)
    st = _on_device_of(w, colibri_moe_quantize_fp8, w.data_ptr(), rows, cols, codes.data_ptr(), scales.data_ptr(),
                       _stream_of(w, stream))
    if stream is not None:
        w.record_stream(stream)
    if st != OK:
        raise ColibriError("colibri_moe_quantize_fp8", st)
    return codes, scales


def colibri_moe_quantize_mxfp4(w_ptr: int, dtype: int, rows: int, cols: int, row_stride: int, codes_ptr: int,
                               scales_ptr: int, hip_stream: int = 0) -> int:
    return lib().colibri_moe_quantize_mxfp4(w_ptr, dtype, rows, cols, row_stride, codes_ptr, scales_ptr, hip_stream)


def colibri_moe_dequantize_mxfp4(codes_ptr: int, scales_ptr: int, rows: int, cols: int, dtype: int, out_ptr: int,
                                 hip_stream: int = 0) -> int:
    return lib().colibri_moe_dequantize_mxfp4(codes_ptr, scales_ptr, rows, cols, dtype, out_ptr, hip_stream)


def quantize_mxfp4(w, stream=None):
    """(codes uint8 [rows][cols/2], scales uint8 [rows][cols/32]) of a 2-D
    bf16 or fp32 device tensor whose rows are contiguous (they may be slices of
    longer ones): the 4-bit microscaled codes a layer built with
    FLAG_MXFP4_WEIGHTS keeps. cols must be a multiple of 32. The work is
    enqueued on `stream`, by default the current one; a given stream must
    already be ordered behind the work that makes w."""
    import torch

    bf16 = w.dtype == torch.bfloat16
    if not (bf16 or w.dtype == torch.float32) or w.dim() != 2 or not w.is_cuda:
        raise TypeError("w must be a 2-D bfloat16 or float32 device tensor")
    rows, cols = w.shape
    row_stride, step = w.stride()
    if cols % 32 != 0 or (cols > 1 and step != 1) or (rows > 1 and row_stride < cols):
        raise ValueError("rows must be contiguous, a multiple of 32 long, and must not overlap")
    if stream is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=w.device)
        scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=w.device)
    else:
        empty = _empty_on(stream, w.device)
        codes, scales = empty((rows, cols // 2), torch.uint8), empty((rows, cols // 32), torch.uint8)
    if rows == 0 or cols == 0:
        return codes, scales
    st = _on_device_of(w, colibri_moe_quantize_mxfp4, w.data_ptr(), BF16 if bf16 else F32, rows, cols,
                       row_stride if rows > 1 else cols, codes.data_ptr(), scales.data_ptr(), _stream_of(w, stream))
    if stream is not None:  # w's memory is not used again before this stream is done with it
        w.record_stream(stream)
    if st != OK:
        raise ColibriError("colibri_moe_quantize_mxfp4", st)
    return codes, scales


def dequantize_mxfp4(codes, scales, dtype=None, stream=None):
    """The values [rows][cols] (bf16 by default, or fp32) of 4-bit microscaled
    rows: contiguous uint8 device tensors codes [rows][cols/2] and scales
    [rows][cols/32]. Exact. The work is enqueued on `stream`, by default the
    current one; a given stream must already be ordered behind the work that
    makes the codes and scales."""
    import torch

    bf16 = dtype is None or dtype == torch.bfloat16
    if not (bf16 or dtype == torch.float32):
        raise TypeError("dtype must be bfloat16 or float32")
    for t in (codes, scales):
        if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
            raise TypeError("codes and scales must be contiguous 2-D uint8 device tensors")
    rows, cols = codes.shape[0], codes.shape[1] * 2
    if scales.device != codes.device or scales.shape[0] != rows or scales.shape[1] * 32 != cols:
        raise ValueError("codes [rows][cols/2] and scales [rows][cols/32] do not belong together")
    value = torch.bfloat16 if bf16 else torch.float32
    if stream is None:
        out = torch.empty((rows, cols), dtype=value, device=codes.device)
    else:
        out = _empty_on(stream, codes.device)((rows, cols), value)
    if rows == 0 or cols == 0:
        return out
    st = _on_device_of(codes, colibri_moe_dequantize_mxfp4, codes.data_ptr(), scales.data_ptr(), rows, cols,
                       BF16 if bf16 else F32, out.data_ptr(), _stream_of(codes, stream))
    if stream is not None:
        for t in (codes, scales):
            t.record_stream(stream)
    if st != OK:
        raise ColibriError("colibri_moe_dequantize_mxfp4", st)
    return out


class RoutingRule:
    """How experts are chosen and weighted from logits (colibri_moe_rule_t):
    scoring "softmax" (over all experts) or "sigmoid"; the experts in `groups`
    equal consecutive groups, of which the `top_groups` (default: all) with the
    largest group_score stay, "max" (their best expert) or "top2" (the sum of
    their two best); the weights of a token divided by their sum if normalize,
    then multiplied by scale. The default is the softmax over the k largest
    logits."""

    def __init__(self, scoring="softmax", groups=1, top_groups=None, group_score="max", normalize=True, scale=1.0):
        if scoring not in ("softmax", "sigmoid"):
            raise ValueError('scoring must be "softmax" or "sigmoid"')
        if group_score not in ("max", "top2"):
            raise ValueError('group_score must be "max" or "top2"')
        top_groups = groups if top_groups is None else top_groups
        if max(abs(groups), abs(top_groups)) > _I32_MAX:
            raise ValueError("at most 64 groups")
        self.c = Rule(int(scoring == "sigmoid"), groups, top_groups, int(group_score == "top2"), int(bool(normalize)),
                      scale)


_default_rule = RoutingRule()


def colibri_moe_route(logits_ptr: int, dtype: int, row_stride: int, T: int, E: int, k: int, rule: Rule, bias_ptr,
                      ids_ptr: int, weights_ptr: int, hip_stream: int = 0) -> int:
    return lib().colibri_moe_route(logits_ptr, dtype, row_stride, T, E, k, None if rule is None else ctypes.byref(rule),
                                   bias_ptr, ids_ptr, weights_ptr, hip_stream)


def _check_select_bias(bias, E, device):
    import torch

    if bias.dtype != torch.float32 or bias.device != device or not bias.is_contiguous() or bias.numel() != E:
        raise TypeError("the selection bias must be a contiguous float32 tensor of E values on the same device")


def route(logits, top_k, rule: RoutingRule | None = None, bias=None, stream=None):
    """(ids int32 [T][top_k], weights fp32 [T][top_k]) of router logits [T][E],
    a bf16 or fp32 device tensor with contiguous rows (they may be slices of
    longer ones), by a RoutingRule; bias [E] fp32 is added to the scores for the
    choice alone. At most 256 experts, top_k at most 8. The work is enqueued on
    `stream`, by default the current one; a given stream must already be
    ordered behind the work that makes the tensors."""
    import torch

    bf16 = logits.dtype == torch.bfloat16
    if not (bf16 or logits.dtype == torch.float32) or logits.dim() != 2 or not logits.is_cuda:
        raise TypeError("logits must be a 2-D bfloat16 or float32 device tensor")
    T, E = logits.shape
    if T > _I32_MAX or E > _I32_MAX or top_k > _I32_MAX:
        raise ColibriError("colibri_moe_route", ERR_INVALID_ARG)
    row_stride, step = logits.stride()
    if (E > 1 and step != 1) or (T > 1 and row_stride < E):
        raise ValueError("rows must be contiguous and must not overlap")
    if bias is not None:
        _check_select_bias(bias, E, logits.device)
    if stream is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=logits.device)
        weights = torch.empty((T, top_k), dtype=torch.float32, device=logits.device)
    else:
        empty = _empty_on(stream, logits.device)
        ids, weights = empty((T, top_k), torch.int32), empty((T, top_k), torch.float32)
        for t in (logits, bias):
            if t is not None:
                t.record_stream(stream)
    st = _on_device_of(logits, colibri_moe_route, logits.data_ptr(), BF16 if bf16 else F32, row_stride if T > 1 else E,
                       T, E, top_k, (rule or _default_rule).c, None if bias is None else bias.data_ptr(),
                       ids.data_ptr(), weights.data_ptr(), _stream_of(logits, stream))
    if st != OK:
        raise ColibriError("colibri_moe_route", st)
    return ids, weights


def colibri_moe_rms_norm(norm: Norm, hip_stream: int = 0) -> int:
    return lib().colibri_moe_rms_norm(None if norm is None else ctypes.byref(norm), hip_stream)


class Normed(NamedTuple):
    """Outputs of rms_norm; None where a call has none."""

    y: object
    residual: object
    codes: object
    scales: object


def _row_stride(t, name):
    """Row stride of a 2-D tensor whose rows are contiguous."""
    rows, cols = t.shape
    stride, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and stride < cols):
        raise ValueError(f"rows of {name} must be contiguous and must not overlap")
    return stride if rows > 1 else cols


def _rows_of(t, like, name):
    """Row stride of a 2-D device tensor that fits `like`."""
    if t.dtype != like.dtype or t.shape != like.shape or t.device != like.device:
        raise TypeError(f"{name} must have the shape, dtype and device of x")
    return _row_stride(t, name)


def rms_norm(x, weight, eps=1e-6, residual=None, quantize=None, with_y=True, y=None, residual_out=None, stream=None):
    """Root-mean-square norm of the rows of x [T][d] (bf16 or fp32, rows
    contiguous, they may be slices of longer ones) with weight [d] (x's dtype or
    fp32), of x + residual if a residual of the same shape is given:
    Normed(y, residual, codes, scales) with residual = x + residual. quantize
    "fp8" also gives y's E4M3 codes (uint8) and power-of-two row scales, in
    quantize_fp8's format, from the unrounded values; with_y=False leaves y out.
    Given outputs y (contiguous) and residual_out are written and returned; each
    may be x or residual itself, and may not overlap anything else. The work is enqueued on `stream`, by default the
    current one; a given stream must already be ordered behind the work that
    makes the tensors."""
    import torch

    bf16 = x.dtype == torch.bfloat16
    if not (bf16 or x.dtype == torch.float32) or x.dim() != 2 or not x.is_cuda:
        raise TypeError("x must be a 2-D bfloat16 or float32 device tensor")
    T, d = x.shape
    if d > _I32_MAX:
        raise ColibriError("colibri_moe_rms_norm", ERR_INVALID_ARG)
    x_stride = _row_stride(x, "x")
    w_bf16 = weight.dtype == torch.bfloat16
    if not (w_bf16 and bf16 or weight.dtype == torch.float32) or weight.device != x.device or weight.dim() != 1:
        raise TypeError("weight must be a 1-D tensor of x's dtype or float32 on x's device")
    if weight.shape[0] != d or not weight.is_contiguous():
        raise ValueError("weight must be contiguous and hold d values")
    if quantize not in (None, "fp8"):
        raise ValueError('quantize must be None or "fp8"')
    if y is not None and (y.dtype != x.dtype or y.shape != x.shape or y.device != x.device
                          or not y.is_contiguous()):
        raise TypeError("y must be a contiguous tensor of x's shape, dtype and device")
    r_stride = _rows_of(residual, x, "residual") if residual is not None else d
    if residual_out is not None and residual is None:
        raise ValueError("residual_out without a residual")
    ro_stride = _rows_of(residual_out, x, "residual_out") if residual_out is not None else d
    if not with_y and y is not None:
        raise ValueError("y given with with_y=False")
    if not with_y and quantize is None and residual is None:
        raise ValueError("nothing to compute")
    if stream is None:
        def empty(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=x.device)
    else:
        empty = _empty_on(stream, x.device)
        for t in (x, weight, residual, y, residual_out):
            if t is not None:
                t.record_stream(stream)
    like = stream is None and x.is_contiguous()  # the cheaper allocation
    if with_y and y is None:
        y = torch.empty_like(x) if like else empty((T, d), x.dtype)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(x) if like else empty((T, d), x.dtype)
    codes = scales = None
    if quantize is not None:
        codes, scales = empty((T, d), torch.uint8), empty((T,), torch.float32)
    out = Normed(y, residual_out, codes, scales)
    if T == 0 or d == 0:
        if T > 0 and scales is not None:  # rows of no values have the scale of rows of zeros
            with torch.cuda.stream(stream):  # None: where we are
                scales.fill_(1.0)
        return out
    n = Norm(x.data_ptr(), x_stride, None if residual is None else residual.data_ptr(), r_stride, weight.data_ptr(),
             BF16 if bf16 else F32, BF16 if w_bf16 else F32, T, d, eps, None if y is None else y.data_ptr(),
             None if residual is None else residual_out.data_ptr(), ro_stride,
             None if codes is None else codes.data_ptr(), None if codes is None else scales.data_ptr())
    st = _on_device_of(x, colibri_moe_rms_norm, n, _stream_of(x, stream))
    if st != OK:
        raise ColibriError("colibri_moe_rms_norm", st)
    return out


def colibri_moe_quantize_int4(w_ptr: int, dtype: int, rows: int, cols: int, row_stride: int, group: int, codes_ptr: int,
                              scales_ptr: int, zeros_ptr, hip_stream: int = 0) -> int:
    return lib().colibri_moe_quantize_int4(w_ptr, dtype, rows, cols, row_stride, group, codes_ptr, scales_ptr, zeros_ptr,
                                           hip_stream)


def colibri_moe_dequantize_int4(codes_ptr: int, scales_ptr: int, scale_dtype: int, zeros_ptr, rows: int, cols: int,
                                group: int, dtype: int, out_ptr: int, hip_stream: int = 0) -> int:
    return lib().colibri_moe_dequantize_int4(codes_ptr, scales_ptr, scale_dtype, zeros_ptr, rows, cols, group, dtype,
                                             out_ptr, hip_stream)


def colibri_moe_int4_bytes(m: Int4) -> int:
    return lib().colibri_moe_int4_bytes(None if m is None else ctypes.byref(m))


def colibri_moe_int4_pack(m: Int4, codes_ptr: int, scales_ptr: int, zeros_ptr, packed_ptr: int,
                          hip_stream: int = 0) -> int:
    return lib().colibri_moe_int4_pack(None if m is None else ctypes.byref(m), codes_ptr, scales_ptr, zeros_ptr,
                                       packed_ptr, hip_stream)


def colibri_moe_int4_linear(m: Int4, packed_ptr: int, x_ptr: int, T: int, k: int, x_per_slot: int, ids_ptr, weights_ptr,
                            y_ptr: int, y_dtype: int, hip_stream: int = 0) -> int:
    return lib().colibri_moe_int4_linear(None if m is None else ctypes.byref(m), packed_ptr, x_ptr, T, k, x_per_slot,
                                         ids_ptr, weights_ptr, y_ptr, y_dtype, hip_stream)


def quantize_int4(w, group=128, symmetric=False, stream=None):
    """(codes uint8 [..][K/2], scales bf16 [..][K/group], zeros uint8 or None) of
    a bf16 or fp32 device tensor w, [N][K] with contiguous rows (they may be
    slices of longer ones) or a contiguous [E][N][K]: 4-bit codes of groups of
    `group` values (32, 64 or a multiple of 128, dividing K), each with a scale
    and a zero point (symmetric: none, codes around 8). The work is enqueued on
    `stream`, by default the current one; a given stream must already be
    ordered behind the work that makes w."""
    import torch

    bf16 = w.dtype == torch.bfloat16
    if not (bf16 or w.dtype == torch.float32) or w.dim() not in (2, 3) or not w.is_cuda:
        raise TypeError("w must be a 2-D or 3-D bfloat16 or float32 device tensor")
    *lead, cols = w.shape
    rows = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    row_stride = cols
    if len(lead) == 1:
        stride, step = w.stride()
        if (cols > 1 and step != 1) or (rows > 1 and stride < cols):
            raise ValueError("rows must be contiguous and must not overlap")
        row_stride = stride if rows > 1 else cols
    elif not w.is_contiguous():
        raise ValueError("a 3-D w must be contiguous")
    if group not in (32, 64) and (group <= 0 or group % 128 != 0) or cols % group != 0:
        raise ValueError("group must be 32, 64 or a multiple of 128, and divide the row length")
    if stream is None:
        def empty(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=w.device)
    else:
        empty = _empty_on(stream, w.device)
        w.record_stream(stream)
    codes = empty((*lead, cols // 2), torch.uint8)
    scales = empty((*lead, cols // group), torch.bfloat16)
    zeros = None if symmetric else empty((*lead, cols // group), torch.uint8)
    if rows == 0 or cols == 0:
        return codes, scales, zeros
    st = _on_device_of(w, colibri_moe_quantize_int4, w.data_ptr(), BF16 if bf16 else F32, rows, cols, row_stride, group,
                       codes.data_ptr(), scales.data_ptr(), None if zeros is None else zeros.data_ptr(),
                       _stream_of(w, stream))
    if st != OK:
        raise ColibriError("colibri_moe_quantize_int4", st)
    return codes, scales, zeros


def _int4_group(codes, scales, zeros):
    """Group length of matching contiguous device tensors of 4-bit groups."""
    import torch

    if codes.dtype != torch.uint8 or codes.dim() not in (2, 3) or not codes.is_cuda or not codes.is_contiguous():
        raise TypeError("codes must be a contiguous 2-D or 3-D uint8 device tensor")
    if (scales.dtype not in (torch.bfloat16, torch.float16) or scales.device != codes.device
            or not scales.is_contiguous()):
        raise TypeError("scales must be a contiguous bfloat16 or float16 tensor on the codes' device")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.device != codes.device or not zeros.is_contiguous()):
        raise TypeError("zeros must be a contiguous uint8 tensor on the codes' device")
    cols, groups = codes.shape[-1] * 2, scales.shape[-1] if scales.dim() else 0
    if (tuple(scales.shape[:-1]) != tuple(codes.shape[:-1]) or groups == 0 or cols % groups != 0
            or (zeros is not None and tuple(zeros.shape) != tuple(scales.shape))):
        raise ValueError("codes [..][K/2], scales and zeros [..][K/group] do not belong together")
    return cols // groups


def dequantize_int4(codes, scales, zeros=None, dtype=None, stream=None):
    """The values [..][K] (bf16 by default, rounded; or fp32, exact) of 4-bit
    groups as quantize_int4 gives them (scales bf16 or fp16; of a zero point's
    byte the low four bits count, without zeros every zero point is 8): what
    MoELayer takes for such weights. The work is enqueued on `stream`, by
    default the current one; a given stream must already be ordered behind the
    work that makes the tensors."""
    import torch

    group = _int4_group(codes, scales, zeros)
    bf16 = dtype is None or dtype == torch.bfloat16
    if not (bf16 or dtype == torch.float32):
        raise TypeError("dtype must be bfloat16 or float32")
    *lead, half = codes.shape
    rows, cols = lead[0] if len(lead) == 1 else lead[0] * lead[1], half * 2
    value = torch.bfloat16 if bf16 else torch.float32
    if stream is None:
        out = torch.empty((*lead, cols), dtype=value, device=codes.device)
    else:
        out = _empty_on(stream, codes.device)((*lead, cols), value)
        for t in (codes, scales, zeros):
            if t is not None:
                t.record_stream(stream)
    if rows == 0:
        return out
    st = _on_device_of(codes, colibri_moe_dequantize_int4, codes.data_ptr(), scales.data_ptr(),
                       BF16 if scales.dtype == torch.bfloat16 else F16, None if zeros is None else zeros.data_ptr(),
                       rows, cols, group, BF16 if bf16 else F32, out.data_ptr(), _stream_of(codes, stream))
    if st != OK:
        raise ColibriError("colibri_moe_dequantize_int4", st)
    return out


class Int4Linear:
    """A matrix of 4-bit groups, or one per expert, laid out once for products
    of few rows (colibri_moe_int4_linear). codes uint8 [N][K/2] or [E][N][K/2],
    scales bf16 or fp16 and zeros uint8 (or None: 8) [..][K/group], as
    quantize_int4 gives them; they are copied. swiglu: the first half of the N
    rows is a gate projection, the second the up projection of the same units.
    The layout is made on `stream`, by default the current one; calls on other
    streams must be ordered behind it."""

    def __init__(self, codes, scales, zeros=None, swiglu: bool = False, stream=None):
        import torch

        group = _int4_group(codes, scales, zeros)
        *lead, half = codes.shape
        self.E, self.N, self.K, self.group = (1 if len(lead) == 1 else lead[0]), lead[-1], half * 2, group
        self.swiglu, self.device = bool(swiglu), codes.device
        self.out_features = self.N // 2 if swiglu else self.N
        n = -1
        if max(self.E, self.N, self.K) <= _I32_MAX:
            self.c = Int4(self.E, self.N, self.K, group, BF16 if scales.dtype == torch.bfloat16 else F16, int(self.swiglu))
            n = colibri_moe_int4_bytes(self.c)
        if n < 0:
            raise ValueError("not supported: K must be a multiple of 32, group 32, 64 or a multiple of 128, E at most 256, "
                             "N even with swiglu")
        if stream is None:
            self.packed = torch.empty((n,), dtype=torch.uint8, device=codes.device)
        else:
            self.packed = _empty_on(stream, codes.device)((n,), torch.uint8)
            for t in (codes, scales, zeros):
                if t is not None:
                    t.record_stream(stream)
        self._home = _stream_of(codes, stream)  # whose pool packed is of
        st = _on_device_of(codes, colibri_moe_int4_pack, self.c, codes.data_ptr(), scales.data_ptr(),
                           None if zeros is None else zeros.data_ptr(), self.packed.data_ptr(), self._home)
        if st != OK:
            raise ColibriError("colibri_moe_int4_pack", st)

    def forward(self, x, ids=None, weights=None, y=None, dtype=None, stream=None):
        """W x for x bf16 [T][K]. With ids (int32 [T][k], one matrix per expert):
        y [T][k][n] for x [T][K] or [T][k][K], or with weights (fp32 [T][k], not
        with swiglu) their weighted sum [T][n]; n is N, or N/2 with swiglu. A slot
        whose id is outside 0..E-1 gives zeros and adds nothing. At most
        INT4_ROWS (128) rows T * k. y bf16, or dtype=torch.float32; a given y is
        written and returned, and may not overlap x, ids or weights. The work is
        enqueued on `stream`, by default the current one; a given stream must
        already be ordered behind the work that makes the tensors."""
        import torch

        if (x.dtype != torch.bfloat16 or not x.is_contiguous() or x.device != self.device or x.dim() not in (2, 3)
                or x.shape[-1] != self.K):
            raise TypeError("x must be a contiguous bfloat16 tensor [T][K] or [T][k][K] on the weights' device")
        T, per_slot, k = x.shape[0], x.dim() == 3, 1
        if ids is not None:
            if ids.dtype != torch.int32 or ids.dim() != 2 or not ids.is_contiguous() or ids.device != self.device:
                raise TypeError("ids must be a contiguous 2-D int32 tensor on the weights' device")
            k = ids.shape[1]
            if ids.shape[0] != T or (per_slot and x.shape[1] != k):
                raise ValueError("ids [T][k] do not fit x")
        elif self.E != 1 or per_slot or weights is not None:
            raise ValueError("one matrix per expert, x [T][k][K] and weights need ids")
        if weights is not None:
            if (weights.dtype != torch.float32 or tuple(weights.shape) != (T, k) or not weights.is_contiguous()
                    or weights.device != self.device):
                raise TypeError("weights must be a contiguous float32 tensor [T][k] on the weights' device")
            if self.swiglu:
                raise ValueError("no weighted sum behind swiglu")
        f32 = dtype == torch.float32
        if not (f32 or dtype is None or dtype == torch.bfloat16):
            raise TypeError("dtype must be bfloat16 or float32")
        shape = (T, self.out_features) if ids is None or weights is not None else (T, k, self.out_features)
        value = torch.float32 if f32 else torch.bfloat16
        if y is not None and (y.dtype != value or tuple(y.shape) != shape or not y.is_contiguous()
                              or y.device != self.device):
            raise TypeError("y must be a contiguous tensor of the result's shape and dtype on the weights' device")
        if T * k > INT4_ROWS:
            raise ColibriError("colibri_moe_int4_linear", ERR_TOO_LARGE)
        if stream is not None:
            _check_stream(stream, self.device)
            for t in (x, ids, weights, y):
                if t is not None:
                    t.record_stream(stream)
        on = _stream_of(x, stream)
        if on != self._home:  # packed is not used again before this stream is done with it
            self.packed.record_stream(stream if stream is not None else torch.cuda.current_stream(self.device))
        if y is None:
            y = (torch.empty(shape, dtype=value, device=self.device) if stream is None
                 else _empty_on(stream, self.device)(shape, value))
        st = _on_device_of(x, colibri_moe_int4_linear, self.c, self.packed.data_ptr(), x.data_ptr(), T, k, int(per_slot),
                           None if ids is None else ids.data_ptr(), None if weights is None else weights.data_ptr(),
                           y.data_ptr(), F32 if f32 else BF16, on)
        if st != OK:
            raise ColibriError("colibri_moe_int4_linear", st)
        return y


def colibri_moe_stream_copy(src_ptr: int, dst_ptr: int, nbytes: int, hip_stream: int = 0) -> int:
    return lib().colibri_moe_stream_copy(ctypes.c_void_p(src_ptr), ctypes.c_void_p(dst_ptr), nbytes,
                                         ctypes.c_void_p(hip_stream))


def stream_copy(src, dst, stream=None):
    """dst <- src with the library's streaming copy kernel (measurement only):
    contiguous device tensors of the same byte size, a multiple of 16."""
    import torch

    if not (src.is_cuda and dst.is_cuda and src.is_contiguous() and dst.is_contiguous()):
        raise TypeError("src and dst must be contiguous device tensors")
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n:
        raise ValueError("src and dst differ in size")
    s = stream if stream is not None else torch.cuda.current_stream()
    st = colibri_moe_stream_copy(src.data_ptr(), dst.data_ptr(), n, s.cuda_stream)
    if st != OK:
        raise ColibriError("colibri_moe_stream_copy", st)


class ColibriError(RuntimeError):
    def __init__(self, where: str, status: int):
        super().__init__(f"{where}: {colibri_moe_status_string(status)} ({status})")
        self.status = status


# --- torch convenience wrapper (device memory and streams only) -------------

class MoELayer:
    """One layer handle with weights copied into the library at construction.

    Weight tensors are CUDA (HIP) tensors: w_router [d][E], b_router [E] fp32 or
    None, w_gate/w_up [E][f][d], w_down [E][d][f], all torch.bfloat16 or all
    torch.float32, on the device the layer is to run on. Its calls run on
    `stream`, by default that device's current one; a given stream must already
    be ordered behind the work that makes the weights. With a rule (RoutingRule,
    select_bias [E] fp32 or None its bias) experts are chosen and weighted by it.
    """

    def __init__(self, w_router, b_router, w_gate, w_up, w_down, top_k: int, max_tokens: int,
                 flags: int = 0, stream=None, rule: RoutingRule | None = None, select_bias=None):
        import torch

        self._torch = torch
        dt = w_router.dtype
        if dt not in (torch.bfloat16, torch.float32):
            raise TypeError("weights must be bfloat16 or float32")
        d, E = w_router.shape
        f = w_gate.shape[1]
        self.d, self.E, self.f, self.k, self.max_tokens = d, E, f, int(top_k), int(max_tokens)
        self.dtype = dt
        if max(d, f, E, abs(self.k), abs(self.max_tokens)) > _I32_MAX:
            raise ColibriError("colibri_moe_init", ERR_INVALID_ARG)
        self.cfg = Config(d, f, E, self.k, self.max_tokens, BF16 if dt == torch.bfloat16 else F32, flags)
        for t in (w_router, w_gate, w_up, w_down):
            if not t.is_cuda or not t.is_contiguous() or t.dtype != dt or t.device != w_router.device:
                raise TypeError("weights must be contiguous tensors of one dtype on one device")
        if (tuple(w_gate.shape), tuple(w_up.shape), tuple(w_down.shape)) != ((E, f, d), (E, f, d), (E, d, f)):
            raise ValueError("w_gate and w_up must be [E][f][d], w_down [E][d][f], for a w_router of [d][E]")
        if b_router is not None and (b_router.dtype != torch.float32 or b_router.device != w_router.device):
            raise TypeError("b_router must be a float32 tensor on the weights' device")
        if b_router is not None and (not b_router.is_contiguous() or b_router.numel() != E):
            raise ValueError("b_router must be contiguous and hold E values")
        wts = Weights(w_router.data_ptr(), None if b_router is None else b_router.data_ptr(),
                      w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr())
        self.device = w_router.device
        if stream is not None:
            _check_stream(stream, self.device)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        if select_bias is not None:
            if rule is None:
                raise ValueError("select_bias without a rule")
            _check_select_bias(select_bias, E, self.device)
        if rule is None:
            st, h = _on_device_of(w_router, colibri_moe_init, self.cfg, wts, self.stream.cuda_stream)
        else:
            st, h = _on_device_of(w_router, colibri_moe_init_rule, self.cfg, wts, rule.c,
                                  None if select_bias is None else select_bias.data_ptr(), self.stream.cuda_stream)
        if st != OK:
            raise ColibriError("colibri_moe_init" if rule is None else "colibri_moe_init_rule", st)
        self.handle = h

    def routing_buffers(self, T: int) -> dict:
        torch = self._torch
        dev = self.device
        A = T * self.k
        return dict(logits=torch.empty(T, self.E, dtype=torch.float32, device=dev),
                    topk_ids=torch.empty(T, self.k, dtype=torch.int32, device=dev),
                    topk_w=torch.empty(T, self.k, dtype=torch.float32, device=dev),
                    expert_counts=torch.empty(self.E, dtype=torch.int32, device=dev),
                    expert_offsets=torch.empty(self.E + 1, dtype=torch.int32, device=dev),
                    perm=torch.empty(A, dtype=torch.int32, device=dev),
                    perm_slot=torch.empty(A, dtype=torch.int32, device=dev),
                    inv=torch.empty(A, dtype=torch.int32, device=dev))

    def forward(self, x, y=None, routing: dict | None = None, static_scratch: bool = False):
        """y [T][d] = layer(x). ``routing`` (from routing_buffers) receives the
        routing outputs; missing keys are not written. Runs on the handle's
        stream, which must already be ordered behind the work that makes x and
        behind earlier uses of a given y or routing buffer. static_scratch: call
        colibri_moe_forward_static (working memory in the library's fixed
        per-GPU array instead of the handle's)."""
        return self._call(colibri_moe_forward_static if static_scratch else colibri_moe_forward, x, y, routing)

    def forward_few(self, x, y=None, routing: dict | None = None):
        """forward for at most FEW_TOKENS tokens in two kernels
        (colibri_moe_forward_few; bf16 layers)."""
        return self._call(colibri_moe_forward_few, x, y, routing)

    def _call(self, fn, x, y, routing):
        torch = self._torch
        if (x.dtype != self.dtype or x.dim() != 2 or x.shape[1] != self.d or not x.is_contiguous()
                or x.device != self.device):
            raise TypeError("x must be a contiguous [T][d] tensor of the layer dtype on the layer's device")
        T = x.shape[0]
        if y is not None and (y.dtype != self.dtype or not y.is_contiguous() or y.device != self.device
                              or y.numel() < T * self.d):
            raise TypeError("y must be a contiguous [T][d] tensor of the layer dtype on the layer's device")
        if routing is not None:
            self._check_routing(routing, T)
        # The kernels run on the handle's stream: when that is not the current
        # one, a y made here is memory of its pool, and the memory of the
        # caller's tensors is not used again before it is done with them.
        other = torch._C._cuda_getCurrentRawStream(x.device.index) != self.stream.cuda_stream
        given = y
        if y is None:
            y = _empty_on(self.stream, x.device)(x.shape, x.dtype) if other else torch.empty_like(x)
        if other:
            for t in (x, given, *((routing or {}).get(n) for n, _ in Routing._fields_)):
                if t is not None:
                    t.record_stream(self.stream)
        r = None
        if routing is not None:
            r = Routing(*[routing[n].data_ptr() if routing.get(n) is not None else None
                          for n, _ in Routing._fields_])
        st = fn(self.handle, x.data_ptr(), T, y.data_ptr(), r)
        if st != OK:
            raise ColibriError(fn.__name__, st)
        return y

    def _check_routing(self, routing, T):
        torch = self._torch
        A, f32, i32 = T * self.k, torch.float32, torch.int32
        for n, dtype, size in (("logits", f32, T * self.E), ("topk_ids", i32, A), ("topk_w", f32, A),
                               ("expert_counts", i32, self.E), ("expert_offsets", i32, self.E + 1),
                               ("perm", i32, A), ("perm_slot", i32, A), ("inv", i32, A)):
            t = routing.get(n)
            if t is not None and (t.dtype != dtype or not t.is_contiguous() or t.device != self.device
                                  or t.numel() < size):
                raise TypeError(f"{n} must be a contiguous {dtype} tensor of {size} elements on the layer's device")

    def stage_times(self) -> dict:
        return dict(zip(STAGES, colibri_moe_stage_times(self.handle)))

    def close(self):
        if getattr(self, "handle", None):
            st = colibri_moe_free(self.handle)
            self.handle = None
            if st != OK:
                raise ColibriError("colibri_moe_free", st)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
