"""Stand-ins for device tensors and streams, for tests of the binding that need
no GPU: each tensor remembers the stream that was current when it was made
(the pool the caching allocator takes its memory from) and the streams it was
recorded on. Nothing is ever read or written."""
import contextlib

import torch


class Stream:
    def __init__(self, handle, index=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", index)


class Tensor:
    is_cuda = True
    _next = 0x10000000

    def __init__(self, shape, dtype, pool, index=0):
        self.shape, self.dtype, self.pool = tuple(shape), dtype, pool
        self.device = torch.device("cuda", index)
        self.recorded = []
        self.ptr = Tensor._next
        Tensor._next += 1 << 24

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for v in self.shape:
            n *= v
        return n

    def stride(self):
        out = [1]
        for v in self.shape[:0:-1]:
            out.insert(0, out[0] * v)
        return tuple(out)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self.ptr

    def record_stream(self, stream):
        self.recorded.append(stream)


class Device:
    """Installs the stand-ins; `made` holds every tensor torch.empty gave out,
    in order, and `current` the current stream."""

    def __init__(self, monkeypatch):
        self.current = Stream(0)
        self.index = 0  # of the current device
        self.made = []

        def empty(*shape, dtype=None, device=None, **_):
            if len(shape) == 1 and not isinstance(shape[0], int):
                shape = shape[0]
            t = Tensor(shape, dtype, self.current, torch.device(device or "cuda").index or 0)
            self.made.append(t)
            return t

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            try:
                yield
            finally:
                self.current = before

        @contextlib.contextmanager
        def device(d):
            before, self.index = self.index, torch.device(d).index
            try:
                yield
            finally:
                self.index = before

        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch, "empty_like", lambda t, **_: empty(t.shape, dtype=t.dtype, device=t.device))
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "current_stream",
                            lambda d=None: self.current if torch.device(d or "cuda").index in (None, 0)
                            else Stream(0x1000, torch.device(d).index))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.index)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda _: self.current.cuda_stream, raising=False)

    def of(self, ptr):
        return next(t for t in self.made if t.ptr == ptr)


def layer(dev, stream=None, dtype=torch.bfloat16, d=64, E=8, f=128, k=2, max_tokens=16):
    """A MoELayer without a handle behind it."""
    import sparse_moe_gemm_amd as cm

    out = cm.MoELayer.__new__(cm.MoELayer)
    out._torch, out.handle, out.dtype, out.device = torch, 0, dtype, torch.device("cuda", 0)
    out.d, out.E, out.f, out.k, out.max_tokens = d, E, f, k, max_tokens
    out.stream = stream if stream is not None else dev.current
    return out
