"""Tensor checks and conversions shared by the bindings."""
from __future__ import annotations

from ._lib import KDA_BF16, KDA_F32, check as lib_check


_torch = None


def torch_module():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


_DT_CODES = {}


def dt_code(dtype):
    code = _DT_CODES.get(dtype)
    if code is None:
        torch = torch_module()
        _DT_CODES.update({torch.bfloat16: KDA_BF16, torch.float32: KDA_F32})
        code = _DT_CODES.get(dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}")
    return code


def ptr(t):
    return 0 if t is None else int(t.data_ptr())


def check(t, name, shape, dtype, device):
    if t is None or (t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous()):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def upstream(grad):
    """A gradient as the kernels take it: autograd may hand over a view of a larger tensor."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


def launch(dev, call, *args):
    """call(*args, stream) with `dev` current, on its current stream; raises on a bad status.  The device is switched only
    where it is another one, and the stream is asked for as its handle: both cost more than the checks of a small call."""
    torch = torch_module()
    index = dev.index
    if index == torch.cuda.current_device():
        status = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = call(*args, _raw_stream(index))
    if status:
        lib_check(status)


def _raw_stream(index):
    global _raw_stream
    torch = torch_module()
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(index)
