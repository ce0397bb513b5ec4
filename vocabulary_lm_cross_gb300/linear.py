"""PyTorch-facing binding of the linear layer and the gated feed-forward layer
(argument marshalling only): linear_fwd / linear_bwd and glu_fwd / glu_bwd of
libvlmce.so."""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import capi
from .rows import (ACTS, DTYPES, current_device, matrix, raw_stream, rows, vector,
                   workspace_of)

_FP8 = torch.float8_e4m3fn


class LinearResult(NamedTuple):
    y: torch.Tensor              # [T, N]
    preact: torch.Tensor | None  # [T, N] (gated: [T, 2n]), where asked for


class LinearGrads(NamedTuple):
    dx: torch.Tensor | None
    dweight: torch.Tensor | None
    dbias: torch.Tensor | None   # fp32 [N]


class LinearPlan(NamedTuple):
    """vlmce_linear_describe_plan in include/vlmce.h says what the fields are."""
    kernel: str       # "pairs" or "small"
    outputs: int
    tokens: int
    split: int
    tiles: int
    dealt: bool
    per_sm: int
    exchanges: int


def describe_linear_plan(T: int, N: int, K: int, dtype: torch.dtype, *, gated: bool = False,
                         backward: bool = False) -> LinearPlan:
    """The kernels that a linear (gated: glu) layer runs for these sizes on the current
    device; backward: those of its gradients."""
    out = (ctypes.c_int32 * 8)()
    capi.check(capi.lib().vlmce_linear_describe_plan(int(gated), int(backward), T, N, K, DTYPES[dtype],
                                                     ctypes.cast(out, ctypes.c_void_p)),
               "vlmce_linear_describe_plan")
    return LinearPlan(("pairs", "small")[out[0]], out[1], out[2], out[3], out[4], bool(out[5]), out[6],
                      out[7])


def _act(act: str, gated: bool) -> int:
    if act not in ACTS or (gated and act == "none"):
        raise ValueError(f"act must be one of {[a for a in ACTS if not gated or a != 'none']}")
    return ACTS[act]


def _operands(x, weight):
    matrix(x, "x")
    matrix(weight, "weight")
    dt = x.dtype
    if dt not in DTYPES or dt == torch.float32:
        raise TypeError("x must be bf16, fp16 or float8_e4m3fn")
    return (dt, rows(x, "x", x.shape, dt, x.device),
            rows(weight, "weight", (weight.shape[0], x.shape[1]), dt, x.device))


def _forward(gated, x, weight, bias, residual, act, preact, x_scale, weight_scale, out_dtype, out,
             dev_err):
    dt, xs, ws = _operands(x, weight)
    dev = x.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return _forward(gated, x, weight, bias, residual, act, preact, x_scale, weight_scale,
                            out_dtype, out, dev_err)
    T, K = x.shape
    R = weight.shape[0]
    a = _act(act, gated)
    if gated and R % 2:
        raise ValueError("weight must have 2n rows")
    N = R // 2 if gated else R
    xsc = wsc = None
    if dt == _FP8:
        odt = out_dtype or torch.bfloat16
        if x_scale is None or weight_scale is None:
            raise ValueError("float8_e4m3fn operands need x_scale and weight_scale")
        xsc = vector(x_scale, "x_scale", T, (torch.float32,), dev)
        wsc = vector(weight_scale, "weight_scale", R, (torch.float32,), dev)
    else:
        odt = out_dtype or dt
        if x_scale is not None or weight_scale is not None:
            raise ValueError("x_scale and weight_scale go with float8_e4m3fn operands")
    if odt not in (torch.bfloat16, torch.float16) or (dt != _FP8 and odt != dt):
        raise TypeError("out_dtype must be x's dtype, or bf16 or fp16 with float8_e4m3fn operands")
    ys, shape = N, (T, N)
    if out is None:
        out = torch.empty(shape, dtype=odt, device=dev)
    else:
        ys = rows(out, "out", shape, odt, dev)
    z = zp = None
    zs = R
    if preact is True:
        z = torch.empty((T, R), dtype=odt, device=dev)
        zp = z.data_ptr()
    elif preact is not None and preact is not False:
        z = preact
        zs = rows(z, "preact", (T, R), odt, dev)
        zp = z.data_ptr()
    err = None
    if dev_err is not None:
        err = vector(dev_err, "dev_err", 1, (torch.int32,), dev)
    if gated:
        st = capi.lib().glu_fwd(x.data_ptr(), xs, xsc, weight.data_ptr(), ws, wsc, DTYPES[dt],
                                DTYPES[odt], T, N, K, a, out.data_ptr(), ys, zp, zs, err,
                                raw_stream(dev.index))
        if st:
            capi.check(st, "glu_fwd")
        return LinearResult(out, z)
    b = vector(bias, "bias", N, (odt,), dev) if bias is not None else None
    r, rs = None, N
    if residual is not None:
        rs = rows(residual, "residual", shape, odt, dev)
        r = residual.data_ptr()
    st = capi.lib().linear_fwd(x.data_ptr(), xs, xsc, weight.data_ptr(), ws, wsc, DTYPES[dt], b, r,
                               rs, DTYPES[odt], T, N, K, a, out.data_ptr(), ys, zp, zs, err,
                               raw_stream(dev.index))
    if st:
        capi.check(st, "linear_fwd")
    return LinearResult(out, z)


def linear_fwd(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               residual: torch.Tensor | None = None, *, act: str = "none",
               preact: bool | torch.Tensor = False, x_scale: torch.Tensor | None = None,
               weight_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
               out: torch.Tensor | None = None,
               dev_err: torch.Tensor | None = None) -> LinearResult:
    """y = act(x W^T + bias) + residual, x [T, K], weight [N, K].

    bf16 or fp16 operands, or float8_e4m3fn with x_scale [T] and weight_scale
    [N] (fp32).  act: none, silu, gelu, gelu_tanh or relu.  preact: True, or a
    [T, N] tensor, to keep x W^T + bias for linear_bwd.  out may be
    ``residual`` itself.  dev_err: int32 [1] the kernels OR their error bits into;
    without it check_device_errors() tells of them.
    """
    return _forward(False, x, weight, bias, residual, act, preact, x_scale, weight_scale,
                    out_dtype, out, dev_err)


def glu_fwd(x: torch.Tensor, weight: torch.Tensor, *, act: str = "silu",
            preact: bool | torch.Tensor = False, x_scale: torch.Tensor | None = None,
            weight_scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
            out: torch.Tensor | None = None, dev_err: torch.Tensor | None = None) -> LinearResult:
    """y [T, n] = act(x Wg^T) (x Wu^T), weight [2n, K] = (Wg rows | Wu rows).

    act: silu, gelu, gelu_tanh or relu.  preact: True, or a [T, 2n] tensor, to
    keep (x Wg^T | x Wu^T) for glu_bwd.  Other arguments as linear_fwd.
    """
    return _forward(True, x, weight, None, None, act, preact, x_scale, weight_scale, out_dtype,
                    out, dev_err)


def _backward(gated, dy, x, weight, preact, act, bias_grad, want_dx, want_dweight, out, dweight,
              dweight_dtype, dbias, accumulate, workspace, dev_err):
    dt, xs, ws = _operands(x, weight)
    if dt == _FP8:
        raise TypeError("the backward pass takes bf16 or fp16")
    dev = x.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return _backward(gated, dy, x, weight, preact, act, bias_grad, want_dx, want_dweight,
                             out, dweight, dweight_dtype, dbias, accumulate, workspace, dev_err)
    T, K = x.shape
    R = weight.shape[0]
    a = _act(act, gated)
    if gated and R % 2:
        raise ValueError("weight must have 2n rows")
    N = R // 2 if gated else R
    ds = rows(dy, "dy", (T, N), dt, dev)
    z, zs = None, R
    if preact is not None:
        zs = rows(preact, "preact", (T, R), dt, dev)
        z = preact.data_ptr()
    elif act != "none":
        raise ValueError("preact is needed with an activation")
    dxs = K
    if not want_dx:
        if out is not None:
            raise ValueError("out needs want_dx")
    elif out is None:
        out = torch.empty((T, K), dtype=dt, device=dev)
    else:
        dxs = rows(out, "out", (T, K), dt, dev)
    if not want_dweight:
        if dweight is not None:
            raise ValueError("dweight needs want_dweight")
    elif dweight is None:
        if accumulate:
            raise ValueError("accumulate needs dweight")
        dweight = torch.empty((R, K), dtype=dweight_dtype or torch.float32, device=dev)
    if dweight is not None:
        if dweight.shape != (R, K) or not dweight.is_contiguous() or dweight.device != dev or \
                dweight.dtype not in (torch.float32, dt):
            raise ValueError("dweight must be a contiguous [N, K] in fp32 or x's dtype")
        if dweight_dtype is not None and dweight.dtype != dweight_dtype:
            raise TypeError("dweight does not have dweight_dtype")
    b = None
    if bias_grad or dbias is not None:
        if dbias is None:
            if accumulate:
                raise ValueError("accumulate needs dbias")
            dbias = torch.empty(N, dtype=torch.float32, device=dev)
        b = vector(dbias, "dbias", N, (torch.float32,), dev)
    err = None
    if dev_err is not None:
        err = vector(dev_err, "dev_err", 1, (torch.int32,), dev)
    lib = capi.lib()
    need = (lib.vlmce_glu_bwd_workspace_bytes if gated else lib.vlmce_linear_bwd_workspace_bytes)(
        T, N, K)
    # (without an activation and dbias the products read dy itself)
    w = None
    if workspace is not None or a != capi.ACT_NONE or b is not None or ds % 8 or \
            dy.data_ptr() % 16:
        w = workspace_of(workspace, need, dev)
    dw = dweight.data_ptr() if dweight is not None else None
    dwt = DTYPES[dweight.dtype] if dweight is not None else capi.F32
    head = (dy.data_ptr(), ds, x.data_ptr(), xs, weight.data_ptr(), ws, z, zs, DTYPES[dt], T, N, K,
            a, out.data_ptr() if out is not None else None, dxs, dw, dwt)
    tail = (int(accumulate), err, w.data_ptr() if w is not None else None,
            w.numel() * w.element_size() if w is not None else 0, raw_stream(dev.index))
    if gated:
        capi.check(lib.glu_bwd(*head, *tail), "glu_bwd")
    else:
        capi.check(lib.linear_bwd(*head, b, *tail), "linear_bwd")
    return LinearGrads(out, dweight, dbias)


def linear_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
               preact: torch.Tensor | None = None, *, act: str = "none", bias_grad: bool = False,
               want_dx: bool = True, want_dweight: bool = True, out: torch.Tensor | None = None,
               dweight: torch.Tensor | None = None, dweight_dtype: torch.dtype | None = None,
               dbias: torch.Tensor | None = None, accumulate: bool = False,
               workspace: torch.Tensor | None = None,
               dev_err: torch.Tensor | None = None) -> LinearGrads:
    """Gradients of linear_fwd (bf16 or fp16): dx, dweight (fp32 unless
    dweight_dtype, x's dtype, asks otherwise) and, with bias_grad or dbias, dbias
    (fp32).  The residual's gradient is dy.  accumulate: add to the given fp32
    dweight and dbias.  The gradient of the pre-activations is rounded to x's dtype:
    in fp16 it must stay within 65504."""
    return _backward(False, dy, x, weight, preact, act, bias_grad, want_dx, want_dweight, out,
                     dweight, dweight_dtype, dbias, accumulate, workspace, dev_err)


def glu_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, preact: torch.Tensor, *,
            act: str = "silu", want_dx: bool = True, want_dweight: bool = True,
            out: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
            dweight_dtype: torch.dtype | None = None, accumulate: bool = False,
            workspace: torch.Tensor | None = None,
            dev_err: torch.Tensor | None = None) -> LinearGrads:
    """Gradients of glu_fwd (bf16 or fp16): dx [T, K] and dweight [2n, K] (fp32
    unless dweight_dtype, x's dtype, asks otherwise); dbias is None.  The range of
    fp16 as in linear_bwd."""
    return _backward(True, dy, x, weight, preact, act, False, want_dx, want_dweight, out, dweight,
                     dweight_dtype, None, accumulate, workspace, dev_err)
