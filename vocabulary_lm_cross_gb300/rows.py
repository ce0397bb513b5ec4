"""Argument marshalling shared by the layer bindings (rmsnorm, linear, glu)."""
from __future__ import annotations

import torch

from . import capi

DTYPES = {torch.float32: capi.F32, torch.bfloat16: capi.BF16, torch.float16: capi.F16,
          torch.float8_e4m3fn: capi.E4M3}
ACTS = {"none": capi.ACT_NONE, "silu": capi.ACT_SILU, "gelu": capi.ACT_GELU,
        "gelu_tanh": capi.ACT_GELU_TANH, "relu": capi.ACT_RELU}


def rows(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """The row stride of a 2-D argument, after its checks."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    row, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return row if shape[0] > 1 else shape[1]


def vector(t: torch.Tensor, name: str, n: int, dtypes, device) -> int:
    """The data pointer of a contiguous 1-D argument, after its checks."""
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous [{n}]")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t.data_ptr()


def matrix(t: torch.Tensor, name: str) -> None:
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")


# The current device and the handle of its current stream.  torch.cuda's functions
# for these check for lazy initialisation (a CUDA tensor exists here) and build a
# Stream object, 2 us a call on the host.
current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if raw_stream is None:  # a CPU-only torch
    def raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def workspace_of(workspace, need: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace
