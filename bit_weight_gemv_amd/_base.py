"""What the bindings of the experts' and the adapters' entry points share."""
from __future__ import annotations

_functions = {}


def torch_module():
    import torch
    return torch


def function(name, table):
    """The entry point `name` of the loaded library with its argument types
    (those of `table`) set."""
    import bit_weight_gemv_amd as q4
    L = q4.lib()
    f = _functions.get(name)
    if f is None or f[0] is not L:
        g = getattr(L, name)
        g.argtypes, g.restype = table[name]
        f = _functions[name] = (L, g)
    return f[1]


def check(t, name, dtype, device):
    import bit_weight_gemv_amd as q4
    q4._check(t, name, dtype, device)


def out_type(dtype, name):
    import bit_weight_gemv_amd as q4
    torch = torch_module()
    if dtype == torch.bfloat16:
        return q4.Q4_OUT_BF16
    if dtype == torch.float32:
        return q4.Q4_OUT_F32
    raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")


class on:
    """The call's device and stream, made current while outputs and scratch
    are allocated and the work is enqueued: a new tensor then belongs to the
    stream that writes it, and scratch goes back to that stream's memory.
    stream None: the device's current one."""

    def __init__(self, device, stream):
        torch = torch_module()
        if device.type != "cuda":
            raise ValueError(f"the tensors must be on a GPU, got {device}")
        self.device, self.guard = device, None
        here = torch.cuda.current_device() == device.index
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                handle = int(stream)
                stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
            if stream.device != device:
                raise ValueError(f"the stream must be on {device}, got {stream.device}")
            if not here or stream.cuda_stream != torch.cuda.current_stream().cuda_stream:
                self.guard = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream
        else:
            if not here:
                self.guard = torch.cuda.device(device)
            self.handle = torch.cuda.current_stream(device).cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *e):
        if self.guard is not None:
            self.guard.__exit__(*e)
        return False

    def output(self, t, shape, dtype, name):
        """The caller's output tensor, checked, or a new one."""
        if t is None:
            return torch_module().empty(shape, dtype=dtype, device=self.device)
        check(t, name, dtype, self.device)
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        return t

    def workspace(self, given, need):
        """(pointer, bytes) of the caller's workspace, or of a new one that
        lives until the call has enqueued its work."""
        if given is not None:
            check(given, "workspace", torch_module().uint8, self.device)
            return given.data_ptr(), given.numel()
        if need == 0:
            return None, 0
        self.kept = torch_module().empty(need, dtype=torch_module().uint8, device=self.device)
        return self.kept.data_ptr(), need


def raise_for(status, name):
    import bit_weight_gemv_amd as q4
    if status != q4.Q4_OK:
        raise q4.Q4Error(status, name)
