"""What the bindings of the experts' and the adapters' entry points share.
The smallest calls take a few microseconds on the GPU, so nothing here is
looked up twice."""
from __future__ import annotations

import functools

_torch = None
_functions = {}
_q4 = None


def torch_module():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _package():
    global _q4
    if _q4 is None:
        import bit_weight_gemv_amd
        _q4 = bit_weight_gemv_amd
    return _q4


def function(name, table):
    """The entry point `name` of the loaded library with its argument types
    (those of `table`) set."""
    q4 = _q4 or _package()
    f = _functions.get(name)
    if f is None or f[0] is not q4._lib:
        L = q4.lib()
        g = getattr(L, name)
        g.argtypes, g.restype = table[name]
        f = _functions[name] = (L, g)
    return f[1]


def sizes(f):
    """A size that depends on the shape alone, kept for the next call."""
    return functools.lru_cache(maxsize=4096)(f)


def check(t, name, dtype, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def out_type(dtype, name):
    torch = _torch or torch_module()
    if dtype == torch.bfloat16:
        return 1  # Q4_OUT_BF16
    if dtype == torch.float32:
        return 0  # Q4_OUT_F32
    raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")


class on:
    """The call's device and stream, made current while outputs and scratch
    are allocated and the work is enqueued: a new tensor then belongs to the
    stream that writes it, and scratch goes back to that stream's memory.
    stream None: the device's current one."""

    __slots__ = ("device", "guard", "handle", "kept")

    def __init__(self, device, stream):
        torch = _torch or torch_module()
        if device.type != "cuda":
            raise ValueError(f"the tensors must be on a GPU, got {device}")
        self.device, self.guard, self.kept = device, None, None
        here = torch.cuda.current_device() == device.index
        if stream is None:
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)
            if not here:
                self.guard = torch.cuda.device(device)
            return
        if not hasattr(stream, "cuda_stream"):
            handle = int(stream)
            stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream must be on {device}, got {stream.device}")
        self.handle = stream.cuda_stream
        if not here or self.handle != torch._C._cuda_getCurrentRawStream(device.index):
            self.guard = torch.cuda.stream(stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *e):
        if self.guard is not None:
            return self.guard.__exit__(*e)
        return False

    def output(self, t, shape, dtype, name):
        """The caller's output tensor, checked, or a new one."""
        if t is None:
            return _torch.empty(shape, dtype=dtype, device=self.device)
        check(t, name, dtype, self.device)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        return t

    def workspace(self, given, need):
        """(pointer, bytes) of the caller's workspace, or of a new one that
        lives until the call has enqueued its work."""
        if given is not None:
            check(given, "workspace", _torch.uint8, self.device)
            return given.data_ptr(), given.numel()
        if need == 0:
            return None, 0
        self.kept = _torch.empty(need, dtype=_torch.uint8, device=self.device)
        return self.kept.data_ptr(), need


def raise_for(status, name):
    if status != 0:
        raise _package().Q4Error(status, name)
