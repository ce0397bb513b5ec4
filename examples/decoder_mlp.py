"""The MLP half of a decoder layer and the head, on this library's operators.

Training step (bf16): RMS norm with the residual's addition, gated layer,
closing linear layer with the residual in its epilogue, final norm, fused linear
cross-entropy, and the whole backward pass into fp32 weight gradients.  Serving
step: the same block for a few tokens with the gated layer's weight in e4m3, fed
by the norm's e4m3 output, and the head as a linear layer.

    python examples/decoder_mlp.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocabulary_lm_cross_gb300 as v  # noqa: E402

EPS = 1e-5


class Block:
    """Weights of one block and the head: fp32 masters, bf16 copies for the kernels."""

    def __init__(self, H: int, n: int, V: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def init(*shape, sigma):
            return torch.randn(shape, generator=g, device="cuda") * sigma

        self.master = {"norm": torch.ones(H, device="cuda"), "gate_up": init(2 * n, H, sigma=H ** -0.5),
                       "down": init(H, n, sigma=n ** -0.5), "final": torch.ones(H, device="cuda"),
                       "head": init(V, H, sigma=H ** -0.5)}
        self.sync()

    def sync(self) -> None:
        self.w = {k: t.bfloat16() for k, t in self.master.items()}


def train_step(m: Block, x: torch.Tensor, stream: torch.Tensor, labels: torch.Tensor, lr: float):
    """One SGD step on hidden states x [T, H] and the residual stream [T, H]; the loss."""
    w = m.w
    a = v.rmsnorm_fwd(x, w["norm"], stream, eps=EPS)
    h = v.glu_fwd(a.y, w["gate_up"], preact=True)
    out = v.linear_fwd(h.y, w["down"], residual=a.residual)
    f = v.rmsnorm_fwd(out.y, w["final"], eps=EPS)
    loss = v.flce_fwd_bwd(f.y, w["head"], labels)

    df = v.rmsnorm_bwd(loss.grad_hidden, out.y, w["final"], f.rstd)
    dd = v.linear_bwd(df.dx, h.y, w["down"])
    dh = v.glu_bwd(dd.dx, a.y, w["gate_up"], h.preact)
    # the gradient of the residual stream joins the norm's
    da = v.rmsnorm_bwd(dh.dx, a.residual, w["norm"], a.rstd, dresidual=df.dx)

    grads = {"norm": da.dweight, "gate_up": dh.dweight, "down": dd.dweight, "final": df.dweight,
             "head": loss.grad_weight}
    for k, g in grads.items():
        m.master[k].add_(g, alpha=-lr)
    m.sync()
    return loss.reduced[0]


def quantize_rows(w: torch.Tensor):
    """(e4m3 weight, fp32 scale per row)."""
    w = w.float()
    scale = w.abs().amax(dim=1).clamp(min=1e-30) / 448.0
    return (w / scale[:, None]).to(torch.float8_e4m3fn), scale


class Server:
    """The block for serving: the gated layer's weight in e4m3, laid out once."""

    def __init__(self, m: Block):
        self.w = m.w
        self.gate_up, self.gate_up_scale = quantize_rows(m.w["gate_up"])

    def logits(self, x: torch.Tensor, stream: torch.Tensor) -> torch.Tensor:
        """[T, V] for the hidden states of a few tokens; `stream` is updated in place."""
        a = v.rmsnorm_fwd(x, self.w["norm"], stream, eps=EPS, fp8=True, residual_out=stream)
        h = v.glu_fwd(a.y, self.gate_up, x_scale=a.scale, weight_scale=self.gate_up_scale)
        v.linear_fwd(h.y, self.w["down"], residual=stream, out=stream)
        f = v.rmsnorm_fwd(stream, self.w["final"], eps=EPS)
        return v.linear_fwd(f.y, self.w["head"]).y


def main(T: int = 512, H: int = 256, n: int = 768, V: int = 1000, steps: int = 8):
    m = Block(H, n, V)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    stream = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    losses = [float(train_step(m, x, stream, labels, lr=0.5)) for _ in range(steps)]
    print("loss:", " ".join(f"{v_:.4f}" for v_ in losses))
    # serve single tokens and a batch of them: the same rows either way
    server = Server(m)
    batch = server.logits(x[:4].clone(), stream[:4].clone())
    single = torch.cat([server.logits(x[i:i + 1].clone(), stream[i:i + 1].clone())
                        for i in range(4)])
    v.check_device_errors()  # a program checks where it waits for the GPU anyway
    print("top tokens:", batch.argmax(dim=1).tolist(), "labels:", labels[:4].tolist())
    return losses, batch, single


if __name__ == "__main__":
    main()
