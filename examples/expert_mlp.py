"""A feed-forward layer of experts, on this library's operators in block-scaled e4m3.

Training step: tokens to their experts' rows, both products on operands quantised by
blocks of 128, the experts' results back with the router's weights onto the residual
stream, and the whole backward pass, its products in block-scaled e4m3 too (from the
transposed quantisations), into fp32 weight gradients.  Serving step: the same layer for a
few tokens, quantised on their way to the experts.

    python examples/expert_mlp.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocabulary_lm_cross_gb300 as v  # noqa: E402
from vocabulary_lm_cross_gb300.swiglu import swiglu_bwd, swiglu_fwd  # noqa: E402


class Experts:
    """Weights of E experts: fp32 masters, and their quantisation in blocks of 128 x 128,
    as they are and transposed."""

    def __init__(self, E: int, H: int, n: int, k: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.E, self.k = E, k
        self.router = (torch.randn((E, H), generator=g, device="cuda") * H ** -0.5).bfloat16()
        self.master = {"gate_up": torch.randn((E, 2 * n, H), generator=g, device="cuda") * H ** -0.5,
                       "down": torch.randn((E, H, n), generator=g, device="cuda") * n ** -0.5}
        self.sync()

    def sync(self) -> None:
        self.q = {name: v.quantize_blocks(w, square=True, transposed=True) for name, w in self.master.items()}

    def route(self, x: torch.Tensor):
        """(experts [T, k], their weights fp32 [T, k]) of each token."""
        top = torch.topk(v.linear_fwd(x, self.router).y.float(), self.k, dim=1)
        return top.indices, torch.softmax(top.values, dim=1)


def train_step(m: Experts, x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, dy: torch.Tensor):
    """(y, gradients of x, the weights of the experts, and both matrices) of y = x + experts(x)."""
    up, down = m.q["gate_up"], m.q["down"]
    # an expert's rows start at multiples of 128, so that no block of the transposed
    # quantisations below has two experts' rows
    order = v.moe_sort(experts, m.E, align=128)
    at = order.offsets
    a = v.quantize_blocks(v.moe_gather(x, order).rows, transposed=True)
    z = v.block_linear_fwd(a.q, a.scale, up.q, up.scale, offsets=at)
    h = v.quantize_blocks(swiglu_fwd(z), transposed=True)
    o = v.block_linear_fwd(h.q, h.scale, down.q, down.scale, offsets=at)
    y = v.moe_combine(o, order, weights, residual=x)

    c = v.moe_combine_bwd(dy, o, order, weights)
    d = v.quantize_blocks(c.drows, transposed=True)
    dh = v.block_linear_fwd(d.q, d.scale, down.qt, down.scale_t, offsets=at)
    ddown = v.block_linear_dweight(d.qt, d.scale_t, h.qt, h.scale_t, offsets=at)
    dz = v.quantize_blocks(swiglu_bwd(z, dh), transposed=True)
    da = v.block_linear_fwd(dz.q, dz.scale, up.qt, up.scale_t, offsets=at)
    dup = v.block_linear_dweight(dz.qt, dz.scale_t, a.qt, a.scale_t, offsets=at)
    dx = v.moe_gather_bwd(da, order) + dy
    return y, {"x": dx, "weights": c.dweights, "gate_up": dup, "down": ddown}


def serve(m: Experts, x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
    """The layer for a few tokens; x, the residual stream, is updated in place."""
    order = v.moe_sort(experts, m.E)
    a = v.moe_gather(x, order, fp8=True)
    up, down = m.q["gate_up"], m.q["down"]
    z = v.block_linear_fwd(a.rows, a.scale, up.q, up.scale, offsets=order.offsets)
    h = v.quantize_blocks(swiglu_fwd(z))
    o = v.block_linear_fwd(h.q, h.scale, down.q, down.scale, offsets=order.offsets)
    return v.moe_combine(o, order, weights, residual=x, out=x)


def main(T: int = 512, E: int = 8, k: int = 2, H: int = 256, n: int = 384):
    m = Experts(E, H, n, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    experts, weights = m.route(x)
    y, grads = train_step(m, x, experts, weights, torch.ones_like(x))
    for name in m.master:
        m.master[name].add_(grads[name], alpha=-1e-3)
    m.sync()
    print("tokens of each expert:", torch.bincount(experts.flatten(), minlength=E).tolist())
    print("gradient norms:", {name: round(float(t.float().norm()), 3) for name, t in grads.items()})
    few = serve(m, x[:4].clone(), experts[:4], weights[:4])
    single = torch.cat([serve(m, x[i:i + 1].clone(), experts[i:i + 1], weights[i:i + 1]) for i in range(4)])
    v.check_device_errors()  # a program checks where it waits for the GPU anyway
    print("served rows agree to", float((few.float() - single.float()).norm() / few.float().norm()))
    return y, few, single


if __name__ == "__main__":
    main()
