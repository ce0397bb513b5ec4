"""PyTorch-facing binding of the quantisation by blocks of 128 (argument marshalling
only): quantize_blocks of libvlmce.so."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import capi
from .moe import empty_fp8, padded
from .rows import DTYPES, current_device, raw_stream

_FP8 = torch.float8_e4m3fn


class BlockQuant(NamedTuple):
    """q [.., R, C] and qt [.., C, R] in float8_e4m3fn, their rows whole 16-byte units
    apart; scale and scale_t fp32 with one value for 128 columns (square: and 128 rows)."""
    q: torch.Tensor | None
    scale: torch.Tensor | None
    qt: torch.Tensor | None
    scale_t: torch.Tensor | None


def quantize_blocks(x: torch.Tensor, *, square: bool = False, rows: bool = True,
                    transposed: bool = False) -> BlockQuant:
    """x [R, C] or [E, R, C] (fp32, bf16 or fp16; matrices one behind the other) in
    float8_e4m3fn by blocks of 128.

    rows: q, blocks of 128 columns of a row (what block_linear_fwd takes as x);
    transposed: qt, blocks of 128 rows of a column, transposed (what
    block_linear_dweight takes).  square: blocks of 128 x 128 for either (a weight, and
    the transposed one for the gradient of its inputs)."""
    if x.dim() not in (2, 3):
        raise ValueError("x must have two or three dimensions")
    if not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if x.dtype not in DTYPES or x.dtype == _FP8:
        raise TypeError("x must be fp32, bf16 or fp16")
    if not (rows or transposed):
        raise ValueError("rows or transposed must be asked for")
    dev = x.device
    if dev.index != current_device():
        with torch.cuda.device(dev):
            return quantize_blocks(x, square=square, rows=rows, transposed=transposed)
    *b, R, C = x.shape
    batch = b[0] if b else 1
    if C > 1 and x.stride(-1) != 1:
        raise ValueError("x must have contiguous rows")
    xs = x.stride(-2) if R > 1 else C
    xb = x.stride(0) if b and batch > 1 else 0
    rb, cb = (R + 127) // 128, (C + 127) // 128
    q = s = qt = st_ = None
    if rows:
        q = empty_fp8((*b, R, C), dev)
        s = torch.empty((*b, rb if square else R, cb), dtype=torch.float32, device=dev)
    if transposed:
        qt = empty_fp8((*b, C, R), dev)
        st_ = torch.empty((*b, cb if square else C, rb), dtype=torch.float32, device=dev)
    if x.numel() == 0:
        return BlockQuant(q, s, qt, st_)

    def at(t):
        return t.data_ptr() if t is not None else None

    code = capi.lib().quantize_blocks(x.data_ptr(), DTYPES[x.dtype], batch, R, C, xs, xb,
                                      int(square), at(q), padded(C), at(s), at(qt), padded(R),
                                      at(st_), raw_stream(dev.index))
    if code:
        capi.check(code, "quantize_blocks")
    return BlockQuant(q, s, qt, st_)
