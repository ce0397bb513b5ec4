"""A layer of experts end to end on the GPU: a training step's results and gradients
against the formulas in fp64, without any quantisation, and by differences; a serving step
that gives the same rows for single tokens and for a batch.

An e4m3 value is off by at most 2^-4 of itself, uniformly within its step, so by no more
than 2^-4 / sqrt 3 in the mean; products of many such values, whose errors have no common
sign, are off by as much in norm for each rounded operand, and errors of several operands
add as squares do.  Operands rounded on the way (to y, the router's weights' gradient, the
gradients of down, gate_up and x): x, gate_up, h, down; the same; dy, h, x, gate_up; dy,
down, dz, x and x, gate_up in z; dy, down, dz, gate_up and x, gate_up in z.  So at most six:
sqrt 6 2^-4 / sqrt 3 = 0.089; bf16 roundings (2^-8 each) are within what the rounding up to
0.1 leaves.
"""
import numpy as np
import pytest
import torch

from examples import expert_mlp as ex
from oracle import layers as ol
from tests.layers_parity import f64, gen

pytestmark = pytest.mark.gpu
BOUND = 0.1


def layer(x, experts, weights, gate_up, down):
    """(y, z and h by pair) in fp64."""
    y, kept = x.copy(), {}
    for t, j in np.ndindex(*experts.shape):
        e = int(experts[t, j])
        h, z = ol.glu(x[t:t + 1], gate_up[e])
        y[t] += weights[t, j] * (h @ down[e].T)[0]
        kept[t, j] = (z, h)
    return y, kept


def near(got, want, what):
    err = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert err <= BOUND, (what, err)


@pytest.mark.parametrize("T,E,k,H,n", [(70, 4, 2, 64, 40), (200, 6, 3, 136, 72)])
def test_a_training_step_against_the_formulas(T, E, k, H, n):
    m = ex.Experts(E, H, n, k, seed=T)
    g = gen(T)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    dy = torch.randn((T, H), generator=g).bfloat16().cuda()
    experts, weights = m.route(x)
    experts[experts == 1] = 0  # an expert without rows, and tokens that name one twice
    y, grads = ex.train_step(m, x, experts, weights, dy)
    ids, w = experts.cpu().numpy(), f64(weights)
    up, down = f64(m.master["gate_up"]), f64(m.master["down"])
    want, kept = layer(f64(x), ids, w, up, down)
    near(f64(y) - f64(x), want - f64(x), "y")
    dx, dw = f64(dy).copy(), np.zeros((T, k))
    dup, ddown = np.zeros_like(up), np.zeros_like(down)
    for (t, j), (z, h) in kept.items():
        e = int(ids[t, j])
        d = f64(dy)[t:t + 1]
        dw[t, j] = float((d @ down[e] @ h.T).item())
        d = d * w[t, j]
        ddown[e] += d.T @ h
        dz = ol.glu_dz(d @ down[e], z, "silu")
        dup[e] += dz.T @ f64(x)[t:t + 1]
        dx[t] += (dz @ up[e])[0]
    near(f64(grads["weights"]), dw, "weights")
    near(f64(grads["down"]), ddown, "down")
    near(f64(grads["gate_up"]), dup, "gate_up")
    near(f64(grads["x"]) - f64(dy), dx - f64(dy), "x")
    assert not grads["down"][1].any() and not grads["gate_up"][1].any()

    # along one direction of each matrix, by differences of the fp64 layer (its curvature
    # leaves (1e-4)^2 of it)
    for name, mat in (("gate_up", up), ("down", down)):
        way = torch.randn(mat.shape, generator=g).numpy()
        step = 1e-4
        ends = []
        for sign in (1, -1):
            mats = {"gate_up": up, "down": down}
            mats[name] = mat + sign * step * way
            ends.append(float((layer(f64(x), ids, w, mats["gate_up"], mats["down"])[0] * f64(dy)).sum()))
        slope = (ends[0] - ends[1]) / (2 * step)
        exact = float(((ddown if name == "down" else dup) * way).sum())
        assert abs(slope - exact) <= 1e-6 * max(1.0, np.linalg.norm(ddown if name == "down" else dup) * 10)


def test_the_example_runs_and_serving_agrees_with_itself():
    y, few, single = ex.main(T=150, E=5, k=2, H=136, n=200)
    assert torch.isfinite(y).all()
    # another number of rows may be summed in another order: bf16 steps of 2^-8, and among
    # the e4m3 values of h a few that then round the other way
    rel = (few.float() - single.float()).norm() / few.float().norm()
    assert float(rel) < 2.0 ** -6
