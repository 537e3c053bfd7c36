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

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcolibri_moe.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_OUT_OF_MEMORY, ERR_HIP, ERR_TOO_LARGE = range(7)
STATIC_SCRATCH_BYTES = 64 << 20  # COLIBRI_MOE_STATIC_SCRATCH_BYTES
FEW_TOKENS = 16  # COLIBRI_MOE_FEW_TOKENS
F32, BF16 = 0, 1
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


EXPORTS = ("colibri_moe_init", "colibri_moe_forward", "colibri_moe_forward_static",
           "colibri_moe_forward_few", "colibri_moe_free",
           "colibri_moe_status_string", "colibri_moe_stage_times", "colibri_moe_stage_name",
           "colibri_moe_quantize_fp8", "colibri_moe_quantize_mxfp4", "colibri_moe_dequantize_mxfp4",
           "colibri_moe_stream_copy")

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
    be ordered behind the work that makes the weights.
    """

    def __init__(self, w_router, b_router, w_gate, w_up, w_down, top_k: int, max_tokens: int,
                 flags: int = 0, stream=None):
        import torch

        self._torch = torch
        dt = w_router.dtype
        if dt not in (torch.bfloat16, torch.float32):
            raise TypeError("weights must be bfloat16 or float32")
        d, E = w_router.shape
        f = w_gate.shape[1]
        self.d, self.E, self.f, self.k, self.max_tokens = d, E, f, int(top_k), int(max_tokens)
        self.dtype = dt
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
        st, h = _on_device_of(w_router, colibri_moe_init, self.cfg, wts, self.stream.cuda_stream)
        if st != OK:
            raise ColibriError("colibri_moe_init", st)
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
