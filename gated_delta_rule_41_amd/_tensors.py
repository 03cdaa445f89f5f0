"""Tensor checks and conversions shared by the bindings."""
from __future__ import annotations

from ._lib import KDA_BF16, KDA_F32


def torch_module():
    import torch
    return torch


def dt_code(dtype):
    torch = torch_module()
    if dtype == torch.bfloat16:
        return KDA_BF16
    if dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"unsupported dtype {dtype}")


def ptr(t):
    return 0 if t is None else int(t.data_ptr())


def check(t, name, shape, dtype, device):
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
