"""PyTorch-facing binding of the products of float8_e4m3fn operands with one scale per
block of 128, dense and by experts (argument marshalling only): block_linear_fwd and
block_linear_dweight of libvlmce.so."""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import capi
from .rows import DTYPES, current_device, matrix, raw_stream, rows, vector

_FP8 = torch.float8_e4m3fn


class BlockLinearPlan(NamedTuple):
    """vlmce_block_linear_describe_plan in include/vlmce.h says what the fields are."""
    kernel: str  # "pairs" or "small"
    rows: int
    split: int
    per_stage: int


def describe_block_linear_plan(T: int, N: int, K: int, experts: int | None = None) -> BlockLinearPlan:
    """How block_linear_fwd runs these sizes on the current device."""
    out = (ctypes.c_int32 * 4)()
    capi.check(capi.lib().vlmce_block_linear_describe_plan(
        T, N, K, 1 if experts is None else experts, int(experts is not None), ctypes.cast(out, ctypes.c_void_p)),
        "vlmce_block_linear_describe_plan")
    return BlockLinearPlan(("pairs", "small")[out[0]], out[1], out[2], out[3])


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _stack(t, name, shape, dtype, device):
    """The row stride of [E, rows, cols] whose matrices follow each other."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    stride = rows(t[0], name, shape[1:], dtype, device) if shape[1] > 1 else \
        (t.stride(0) if shape[0] > 1 else shape[2])
    if shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if shape[0] > 1 and t.stride(0) != shape[1] * stride:
        raise ValueError(f"{name}'s matrices must follow each other")
    return stride


def _operand(t, name, device=None):
    if t.dtype is not _FP8:
        raise TypeError(f"{name} must be float8_e4m3fn, not {t.dtype}")
    stride = rows(t, name, t.shape, _FP8, device if device is not None else t.device)
    # (the row stride of a single row is its length, rounded up as a buffer's would be)
    return stride if t.shape[0] > 1 else (stride + 15) // 16 * 16


def _groups(offsets, device):
    if offsets is None:
        return None
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [E + 1]")
    return vector(offsets, "offsets", offsets.shape[0], (torch.int32,), device)


def block_linear_fwd(x: torch.Tensor, x_scale: torch.Tensor, weight: torch.Tensor,
                     weight_scale: torch.Tensor, residual: torch.Tensor | None = None, *,
                     offsets: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                     out: torch.Tensor | None = None,
                     dev_err: torch.Tensor | None = None) -> torch.Tensor:
    """y [T, N] = x W^T (+ residual) of float8_e4m3fn operands with one fp32 scale per
    block of 128 (quantize_blocks, moe_gather).

    x [T, K] with x_scale [T, ceil(K / 128)]; weight [N, K] with weight_scale
    [ceil(N / 128), ceil(K / 128)], or [N, ceil(K / 128)] with a scale for each row.
    offsets (MoEOrder.offsets): weight [E, N, K] and its scales [E, .., ..], rows
    offsets[e] .. offsets[e + 1] of x meet weight[e]; rows behind the last expert's are
    left as they are.  out_dtype: bf16 (unless out or residual say otherwise) or fp16;
    out may be ``residual`` itself.  The gradient of x: dy quantised along its rows with
    the weight's transposed square quantisation.  dev_err as linear_fwd.
    """
    matrix(x, "x")
    dev = x.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return block_linear_fwd(x, x_scale, weight, weight_scale, residual, offsets=offsets,
                                    out_dtype=out_dtype, out=out, dev_err=dev_err)
    xs = _operand(x, "x")
    T, K = x.shape
    kb = _blocks(K)
    off = _groups(offsets, dev)
    if off is None:
        matrix(weight, "weight")
        E, N = 1, weight.shape[0]
        if weight.shape[1] != K:
            raise ValueError(f"weight must be [N, {K}], not {list(weight.shape)}")
        ws = _operand(weight, "weight", dev)
    else:
        E = offsets.shape[0] - 1
        if weight.dim() != 3:
            raise ValueError("with offsets, weight must have three dimensions")
        N = weight.shape[1]
        ws = _stack(weight, "weight", (E, N, K), _FP8, dev)
        if E * N == 1:
            ws = (ws + 15) // 16 * 16
    by_row = weight_scale.dim() >= 2 and weight_scale.shape[-2] == N and N > 1
    sr = N if by_row else _blocks(N)
    if off is None:
        wss = rows(weight_scale, "weight_scale", (sr, kb), torch.float32, dev)
    else:
        wss = _stack(weight_scale, "weight_scale", (E, sr, kb), torch.float32, dev)
    xss = rows(x_scale, "x_scale", (T, kb), torch.float32, dev)
    odt = out_dtype or (out.dtype if out is not None else
                        residual.dtype if residual is not None else torch.bfloat16)
    if odt not in (torch.bfloat16, torch.float16):
        raise TypeError("out_dtype must be bf16 or fp16")
    r, rs, ys = None, N, N
    if residual is not None:
        rs = rows(residual, "residual", (T, N), odt, dev)
        r = residual.data_ptr()
    if out is None:
        out = torch.empty((T, N), dtype=odt, device=dev)
    else:
        ys = rows(out, "out", (T, N), odt, dev)
    err = vector(dev_err, "dev_err", 1, (torch.int32,), dev) if dev_err is not None else None
    st = capi.lib().block_linear_fwd(x.data_ptr(), xs, x_scale.data_ptr(), xss, weight.data_ptr(),
                                     ws, weight_scale.data_ptr(), wss, 1 if by_row else 128, off,
                                     E, r, rs, DTYPES[odt], T, N, K, out.data_ptr(), ys, err,
                                     raw_stream(dev.index))
    if st:
        capi.check(st, "block_linear_fwd")
    return out


def block_linear_dweight(dyt: torch.Tensor, dyt_scale: torch.Tensor, xt: torch.Tensor,
                         xt_scale: torch.Tensor, *, offsets: torch.Tensor | None = None,
                         dweight: torch.Tensor | None = None,
                         dweight_dtype: torch.dtype | None = None, accumulate: bool = False,
                         dev_err: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of block_linear_fwd's weight: dy^T x [N, K] from dyt [N, R] and xt [K, R],
    float8_e4m3fn with a scale per 128 columns (quantize_blocks(.., transposed=True)).

    offsets (moe_sort with align=128): one gradient for each expert, [E, N, K], over its
    columns; without, over all.  fp32 unless dweight or dweight_dtype (bf16, fp16) say
    otherwise; accumulate: add to the given fp32 dweight.  dev_err as linear_fwd."""
    matrix(dyt, "dyt")
    matrix(xt, "xt")
    dev = dyt.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return block_linear_dweight(dyt, dyt_scale, xt, xt_scale, offsets=offsets,
                                        dweight=dweight, dweight_dtype=dweight_dtype,
                                        accumulate=accumulate, dev_err=dev_err)
    ds = _operand(dyt, "dyt")
    xs = _operand(xt, "xt", dev)
    N, R = dyt.shape
    K = xt.shape[0]
    if xt.shape[1] != R:
        raise ValueError(f"xt must be [K, {R}], not {list(xt.shape)}")
    rb = _blocks(R)
    dss = rows(dyt_scale, "dyt_scale", (N, rb), torch.float32, dev)
    xss = rows(xt_scale, "xt_scale", (K, rb), torch.float32, dev)
    off = _groups(offsets, dev)
    shape = (N, K) if off is None else (offsets.shape[0] - 1, N, K)
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate needs dweight")
        dweight = torch.empty(shape, dtype=dweight_dtype or torch.float32, device=dev)
    if dweight.shape != shape or not dweight.is_contiguous() or dweight.device != dev or \
            dweight.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError(f"dweight must be a contiguous {list(shape)} in fp32, bf16 or fp16")
    if dweight_dtype is not None and dweight.dtype != dweight_dtype:
        raise TypeError("dweight does not have dweight_dtype")
    err = vector(dev_err, "dev_err", 1, (torch.int32,), dev) if dev_err is not None else None
    st = capi.lib().block_linear_dweight(dyt.data_ptr(), ds, dyt_scale.data_ptr(), dss,
                                         xt.data_ptr(), xs, xt_scale.data_ptr(), xss, off,
                                         1 if off is None else shape[0], R, N, K,
                                         dweight.data_ptr(), DTYPES[dweight.dtype],
                                         int(accumulate), err, raw_stream(dev.index))
    if st:
        capi.check(st, "block_linear_dweight")
    return dweight
