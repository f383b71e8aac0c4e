"""Checks and conversions shared by the binding's modules: torch tensors to C ABI arguments."""
from __future__ import annotations

import ctypes

import torch

from . import _native


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return _native.WKV_BF16
    if t.dtype == torch.float32:
        return _native.WKV_F32
    raise TypeError(f"unsupported input dtype {t.dtype} (bfloat16 or float32)")


def _dev(t, name, dtype=None, shape=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(ref):
    return ctypes.c_void_p(torch.cuda.current_stream(ref.device).cuda_stream)


def _out_code(y, out_dtype):
    """Output dtype code: that of a given y, else out_dtype (float32 or bfloat16)."""
    dt = y.dtype if y is not None else out_dtype
    if dt == torch.float32:
        return _native.WKV_F32, dt
    if dt == torch.bfloat16:
        return _native.WKV_BF16, dt
    raise TypeError(f"unsupported output dtype {dt} (float32 or bfloat16)")


def _same_dtype(name_tensors):
    dts = {t.dtype for _, t in name_tensors if t is not None}
    if len(dts) != 1:
        raise TypeError("token inputs must share one dtype: " +
                        ", ".join(f"{n}={t.dtype}" for n, t in name_tensors if t is not None))
