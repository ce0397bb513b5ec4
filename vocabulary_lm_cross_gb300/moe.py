"""PyTorch-facing binding of the experts' row operators (argument marshalling only):
moe_sort, moe_gather, moe_combine and their gradients of libvlmce.so."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import capi
from .rows import DTYPES, current_device, matrix, raw_stream, rows

_FP8 = torch.float8_e4m3fn


class MoEOrder(NamedTuple):
    """Where the rows of the experts are (moe_sort)."""
    position: torch.Tensor  # int32 [T, k]: the row of token t's j-th expert, -1: none
    offsets: torch.Tensor   # int32 [E + 1]: where an expert's rows start; the end of the last's
    counts: torch.Tensor    # int32 [E]: its rows in use
    rows: int               # rows of the experts' matrices (any choice of experts fits)


class MoEGather(NamedTuple):
    rows: torch.Tensor           # [order.rows, H] in x's dtype, or float8_e4m3fn
    scale: torch.Tensor | None   # with fp8: fp32 [order.rows, ceil(H / 128)]


class MoECombineGrads(NamedTuple):
    drows: torch.Tensor | None     # [order.rows, H]
    dweights: torch.Tensor | None  # fp32 [T, k]


def moe_sort(experts: torch.Tensor, num_experts: int, *, align: int = 1) -> MoEOrder:
    """The order of tokens by expert: experts [T, k], int32 or int64; ids outside
    [0, num_experts) are nobody's.  An expert's rows follow the order of the tokens
    and start at multiples of ``align`` (block_linear_dweight takes 128)."""
    matrix(experts, "experts")
    if experts.dtype not in (torch.int32, torch.int64):
        raise TypeError("experts must be int32 or int64")
    dev = experts.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return moe_sort(experts, num_experts, align=align)
    T, k = experts.shape
    stride = rows(experts, "experts", experts.shape, experts.dtype, dev)
    E = num_experts if 0 < num_experts <= capi.MOE_MAX_EXPERTS else 1
    position = torch.empty((T, k), dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    st = capi.lib().moe_sort(experts.data_ptr(), stride, int(experts.dtype == torch.int64), T, k,
                      num_experts, align, position.data_ptr(), offsets.data_ptr(),
                      counts.data_ptr(), raw_stream(dev.index))
    if st:
        capi.check(st, "moe_sort")
    # vlmce_moe_rows
    n = (T * k + min(num_experts, T * k) * (align - 1)) // align * align
    return MoEOrder(position, offsets, counts, n)


def _ints(t, name, shape, device):
    if t.shape != shape or t.dtype != torch.int32 or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} on {device}")
    return t.data_ptr()


def _order(order, T, device):
    """(k, E, pointers of position, offsets and counts), after their checks."""
    if order.position.dim() != 2 or order.counts.dim() != 1:
        raise ValueError("order must be moe_sort's")
    k, E = order.position.shape[1], order.counts.shape[0]
    return (k, E, _ints(order.position, "order.position", (T, k), device),
            _ints(order.offsets, "order.offsets", (E + 1,), device),
            _ints(order.counts, "order.counts", (E,), device))


def _dtype(t, name):
    matrix(t, name)
    if t.dtype not in DTYPES or t.dtype == _FP8:
        raise TypeError(f"{name} must be fp32, bf16 or fp16")
    return t.dtype


def _weights(weights, T, k, dt, device):
    """(pointer, stride, dtype) of the tokens' weights."""
    if weights is None:
        return None, k, capi.F32
    if weights.dtype not in (dt, torch.float32):
        raise TypeError(f"weights must be {dt} or fp32")
    return (weights.data_ptr(), rows(weights, "weights", (T, k), weights.dtype, device),
            DTYPES[weights.dtype])


def padded(n: int) -> int:
    """The row stride of an 8-bit matrix of n columns that the products can read."""
    return (n + 15) // 16 * 16


def empty_fp8(shape, device) -> torch.Tensor:
    """An 8-bit tensor of such rows."""
    n = shape[-1]
    if n % 16 == 0:
        return torch.empty(shape, dtype=_FP8, device=device)
    ld = padded(n)
    return torch.empty_strided(shape, (ld, 1) if len(shape) == 2 else (shape[1] * ld, ld, 1),
                               dtype=_FP8, device=device)


def moe_gather(x: torch.Tensor, order: MoEOrder, *, fp8: bool = False,
               out: torch.Tensor | None = None) -> MoEGather:
    """rows[order.position[t, j]] = x[t], x [T, H].  fp8: in float8_e4m3fn with a scale
    per 128 columns (quantize_blocks).  Rows that stand between two experts' become
    zero; those behind the last one's are left as they are."""
    dt = _dtype(x, "x")
    dev = x.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return moe_gather(x, order, fp8=fp8, out=out)
    T, H = x.shape
    xs = rows(x, "x", x.shape, dt, dev)
    k, E, pos, off, cnt = _order(order, T, dev)
    R = order.rows
    odt = _FP8 if fp8 else dt
    if out is None:
        out = empty_fp8((R, H), dev) if fp8 else torch.empty((R, H), dtype=odt, device=dev)
    os_ = rows(out, "out", (R, H), odt, dev)
    scale = torch.empty((R, (H + 127) // 128), dtype=torch.float32, device=dev) if fp8 else None
    st = capi.lib().moe_gather(x.data_ptr(), xs, DTYPES[dt], pos, off, cnt, T, k, E, R, H,
                               out.data_ptr(), os_, DTYPES[odt],
                               scale.data_ptr() if fp8 else None, raw_stream(dev.index))
    if st:
        capi.check(st, "moe_gather")
    return MoEGather(out, scale)


def _combine(data, name, order, weights, residual, out, where):
    dt = _dtype(data, name)
    dev = data.device
    T, H = order.position.shape[0], data.shape[1]
    ds = rows(data, name, (order.rows, H), dt, dev)
    k, _, pos, _, _ = _order(order, T, dev)
    w, ws, wdt = _weights(weights, T, k, dt, dev)
    r, rs, os_ = None, H, H
    if residual is not None:
        rs = rows(residual, "residual", (T, H), dt, dev)
        r = residual.data_ptr()
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=dev)
    else:
        os_ = rows(out, "out", (T, H), dt, dev)
    st = capi.lib().moe_combine(data.data_ptr(), ds, DTYPES[dt], pos, w, ws, wdt, r, rs, T, k,
                                order.rows, H, out.data_ptr(), os_, raw_stream(dev.index))
    if st:
        capi.check(st, where)
    return out


def moe_gather_bwd(drows: torch.Tensor, order: MoEOrder, *,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of moe_gather: dx[t] = sum_j drows[order.position[t, j]]."""
    matrix(drows, "drows")
    if drows.device.index != current_device():
        with torch.cuda.device(drows.device):
            return moe_gather_bwd(drows, order, out=out)
    return _combine(drows, "drows", order, None, None, out, "moe_gather_bwd")


def moe_combine(data: torch.Tensor, order: MoEOrder, weights: torch.Tensor | None = None,
                residual: torch.Tensor | None = None, *,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] data[order.position[t, j]] + residual[t], data [order.rows,
    H] the experts' rows.  weights: [T, k] in fp32 or data's dtype (None: all 1).  out may
    be ``residual`` itself."""
    matrix(data, "data")
    if data.device.index != current_device():
        with torch.cuda.device(data.device):
            return moe_combine(data, order, weights, residual, out=out)
    return _combine(data, "data", order, weights, residual, out, "moe_combine")


def moe_combine_bwd(dy: torch.Tensor, data: torch.Tensor, order: MoEOrder,
                    weights: torch.Tensor | None = None, *, want_drows: bool = True,
                    want_dweights: bool = True, out: torch.Tensor | None = None) -> MoECombineGrads:
    """Gradients of moe_combine: drows (rows that stand between two experts' become
    zero, those behind the last one's are left as they are) and dweights.  The
    residual's gradient is dy."""
    dt = _dtype(dy, "dy")
    dev = dy.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return moe_combine_bwd(dy, data, order, weights, want_drows=want_drows,
                                   want_dweights=want_dweights, out=out)
    T, H = dy.shape
    R = order.rows
    ds = rows(dy, "dy", dy.shape, dt, dev)
    xs = rows(data, "data", (R, H), dt, dev)
    k, E, pos, off, cnt = _order(order, T, dev)
    w, ws, wdt = _weights(weights, T, k, dt, dev)
    os_ = H
    if not want_drows:
        if out is not None:
            raise ValueError("out needs want_drows")
    elif out is None:
        out = torch.empty((R, H), dtype=dt, device=dev)
    else:
        os_ = rows(out, "out", (R, H), dt, dev)
    dw = torch.empty((T, k), dtype=torch.float32, device=dev) if want_dweights else None
    st = capi.lib().moe_combine_bwd(dy.data_ptr(), ds, data.data_ptr(), xs, DTYPES[dt], pos, off,
                                    cnt, w, ws, wdt, T, k, E, R, H,
                                    out.data_ptr() if out is not None else None, os_,
                                    dw.data_ptr() if dw is not None else None,
                                    raw_stream(dev.index))
    if st:
        capi.check(st, "moe_combine_bwd")
    return MoECombineGrads(out, dw)
