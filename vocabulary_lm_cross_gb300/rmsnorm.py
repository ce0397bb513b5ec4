"""PyTorch-facing binding of the RMS norm with the residual's addition
(argument marshalling only): rmsnorm_fwd / rmsnorm_bwd of libvlmce.so."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import capi
from .rows import (DTYPES, current_device, matrix, raw_stream, rows, vector,
                   workspace_of)


class RMSNormResult(NamedTuple):
    y: torch.Tensor                # [T, H] in x's dtype, or float8_e4m3fn
    residual: torch.Tensor | None  # [T, H]: x + residual, what rmsnorm_bwd takes as x (None without a residual)
    rstd: torch.Tensor             # fp32 [T]
    scale: torch.Tensor | None     # fp32 [T] with fp8: y stands for scale[t] y[t]


class RMSNormGrads(NamedTuple):
    dx: torch.Tensor       # [T, H]: gradient of x (and of the residual)
    dweight: torch.Tensor  # fp32 [H]


def _checked(x, weight):
    matrix(x, "x")
    dt = x.dtype
    if dt not in DTYPES or dt == torch.float8_e4m3fn:
        raise TypeError("x must be fp32, bf16 or fp16")
    return dt, vector(weight, "weight", x.shape[1], (dt, torch.float32), x.device)


def rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, *,
                eps: float = 1e-6, weight_offset: float = 0.0, fp8: bool = False,
                out: torch.Tensor | None = None,
                residual_out: torch.Tensor | None = None) -> RMSNormResult:
    """y = s rstd (weight + weight_offset), s = x + residual, per row of x [T, H].

    weight: [H] in x's dtype or fp32.  fp8: y in float8_e4m3fn with one scale
    per row.  residual_out: where s goes (allocated unless given; may be
    ``residual`` or ``x`` itself), only with a residual.
    """
    dt, w = _checked(x, weight)
    dev = x.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return rmsnorm_fwd(x, weight, residual, eps=eps, weight_offset=weight_offset, fp8=fp8,
                               out=out, residual_out=residual_out)
    T, H = shape = x.shape
    xs = rows(x, "x", shape, dt, dev)
    r = ro = None
    rs = ros = H
    if residual is not None:
        rs = rows(residual, "residual", shape, dt, dev)
        r = residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dt, device=dev)
        else:
            ros = rows(residual_out, "residual_out", shape, dt, dev)
        ro = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    ydt = torch.float8_e4m3fn if fp8 else dt
    ys = H
    if out is None:
        out = torch.empty(shape, dtype=ydt, device=dev)
    else:
        ys = rows(out, "out", shape, ydt, dev)
    rstd = torch.empty(T, dtype=torch.float32, device=dev)
    scale = torch.empty(T, dtype=torch.float32, device=dev) if fp8 else None
    st = capi.lib().rmsnorm_fwd(x.data_ptr(), xs, r, rs, w, DTYPES[weight.dtype], DTYPES[dt], T, H,
                                eps, weight_offset, out.data_ptr(), ys, DTYPES[ydt], ro, ros,
                                rstd.data_ptr(), scale.data_ptr() if fp8 else None,
                                raw_stream(dev.index))
    if st:
        capi.check(st, "rmsnorm_fwd")
    return RMSNormResult(out, residual_out, rstd, scale)


def rmsnorm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor, *,
                dresidual: torch.Tensor | None = None, weight_offset: float = 0.0,
                out: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                accumulate_dweight: bool = False,
                workspace: torch.Tensor | None = None) -> RMSNormGrads:
    """Gradients of rmsnorm_fwd.  x: the normalised rows (RMSNormResult.residual,
    or x where there was no residual); dresidual: the gradient reaching them along
    the residual stream.  out: dx (may be ``dy`` or ``dresidual`` itself)."""
    dt, w = _checked(x, weight)
    dev = x.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return rmsnorm_bwd(dy, x, weight, rstd, dresidual=dresidual,
                               weight_offset=weight_offset, out=out, dweight=dweight,
                               accumulate_dweight=accumulate_dweight, workspace=workspace)
    T, H = shape = x.shape
    xs = rows(x, "x", shape, dt, dev)
    ds = rows(dy, "dy", shape, dt, dev)
    rp = vector(rstd, "rstd", T, (torch.float32,), dev)
    dr, drs = None, H
    if dresidual is not None:
        drs = rows(dresidual, "dresidual", shape, dt, dev)
        dr = dresidual.data_ptr()
    os_ = H
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
    else:
        os_ = rows(out, "out", shape, dt, dev)
    if dweight is None:
        if accumulate_dweight:
            raise ValueError("accumulate_dweight needs dweight")
        dweight = torch.empty(H, dtype=torch.float32, device=dev)
    dw = vector(dweight, "dweight", H, (torch.float32,), dev)
    lib = capi.lib()
    ws = workspace_of(workspace, lib.vlmce_rmsnorm_bwd_workspace_bytes(T, H), dev)
    st = lib.rmsnorm_bwd(dy.data_ptr(), ds, x.data_ptr(), xs, w, DTYPES[weight.dtype], rp, dr, drs,
                         DTYPES[dt], T, H, weight_offset, out.data_ptr(), os_, dw,
                         int(accumulate_dweight), ws.data_ptr(),
                         ws.numel() * ws.element_size(),
                         raw_stream(dev.index))
    if st:
        capi.check(st, "rmsnorm_bwd")
    return RMSNormGrads(out, dweight)
