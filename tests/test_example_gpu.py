"""The decoder-layer example end to end on the GPU: a training step's gradients
against the fp64 oracles composed, a falling loss, and a serving step that gives the
same rows for single tokens and for a batch."""
import numpy as np
import pytest
import torch

from examples import decoder_mlp as ex
from oracle import flce as of
from oracle import layers as ol
from tests.layers_parity import f64, gen

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss_and_serving_agrees_with_itself():
    losses, batch, single = ex.main(T=192, H=128, n=264, V=500, steps=6)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    rel = (batch.float() - single.float()).norm() / batch.float().norm()
    assert float(rel) < 2.0 ** -7  # bf16 logits of the same values in another summation order


def test_one_step_against_the_composed_oracles():
    T, H, n, V = 96, 64, 72, 130
    m = ex.Block(H, n, V, seed=3)
    g = gen(4)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    s = torch.randn((T, H), generator=g).bfloat16().cuda()
    labels = torch.randint(0, V, (T,), generator=g).cuda()
    w = {k: f64(t) for k, t in m.w.items()}
    before = {k: t.clone() for k, t in m.master.items()}
    loss = ex.train_step(m, x, s, labels, lr=1.0)

    y1, s1, r1 = ol.rmsnorm(f64(x), w["norm"], f64(s), ex.EPS)
    h, z = ol.glu(y1, w["gate_up"])
    o = ol.linear(h, w["down"], residual=s1)[0]
    y2, _, r2 = ol.rmsnorm(o, w["final"], None, ex.EPS)
    ref = of.flce_fwd_bwd(y2, w["head"], labels.cpu().numpy())
    df, dfinal = ol.rmsnorm_backward(ref["grad_hidden"], o, w["final"], r2)
    dh, ddown, _ = ol.products(df, h, w["down"])
    dy1, dgu, _ = ol.products(ol.glu_dz(dh, z, "silu"), y1, w["gate_up"])
    _, dnorm = ol.rmsnorm_backward(dy1, s1, w["norm"], r1, df)

    assert abs(float(loss) - ref["loss"].mean()) < 2e-2
    for k, want in (("norm", dnorm), ("gate_up", dgu), ("down", ddown), ("final", dfinal),
                    ("head", ref["grad_weight"])):
        got = f64(before[k] - m.master[k])
        # bf16 activations and gradients along the chain: about ten roundings of 2^-8
        assert np.linalg.norm(got - want) <= 10 * 2.0 ** -8 * np.linalg.norm(want), k
