"""Comparison helpers of the decoder-layer GPU tests.

Elementwise bounds, derived from the number formats (u = 2^-8 for bf16 with its 8
significant bits, 2^-11 for fp16, 2^-24 for fp32: half the spacing, relative):

* an output rounded once from fp32: |r - r_o| <= u (|r_o| + e) + tiny + e, with e the
  bound of the fp32 evaluation and tiny the type's smallest step;
* a product sum_k a_k b_k of K terms accumulated in fp32, in any order and with
  truncating or rounding additions: e <= (K + 8) 2^-23 sum_k |a_k b_k|;
* an operand rounded to 16 bits before a product (dz): relative u of each term, so
  e += u sum |dz w| + (subnormals) 2^-25 sum |w| in fp16;
* activations: |act'| <= 1.2, so an error e_z of z gives at most 1.2 e_z, plus a few
  fp32 roundings and the exp2 / reciprocal units' 2^-22: 3e-6 (1 + |z|).
"""
from __future__ import annotations

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U16 = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}
E23 = 2.0 ** -23


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def close(got: torch.Tensor, want: np.ndarray, dtype: str, e, what: str) -> None:
    """Every element within the bound of an output rounded once to dtype."""
    g = f64(got)
    assert g.shape == want.shape, what
    bound = U16[dtype] * (np.abs(want) + e) + TINY[dtype] + e
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[0],
                           g[bad][0], want[bad][0], np.broadcast_to(bound, g.shape)[bad][0])


def randn(g: torch.Generator, shape, dtype, sigma=1.0, pad=0):
    """[rows, cols] (or [n]) ~ N(0, sigma^2) on the GPU, rows padded by `pad` NaNs."""
    v = (torch.randn(shape, generator=g) * sigma).to(dtype)
    if len(shape) == 1 or not pad:
        return v.cuda()
    store = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=dtype)
    store[:, :shape[1]] = v
    return store.cuda()[:, :shape[1]]


def gen(seed: int) -> torch.Generator:
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g
