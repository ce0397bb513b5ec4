"""The fp64 oracle of the decoder-layer operators: closed forms, and every
backward formula against central differences of its forward."""
import numpy as np
import pytest

from oracle import layers as ol

ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]


def diff(f, a, v, h=1e-5):
    return (f(a + h * v) - f(a - h * v)) / (2 * h)


@pytest.mark.parametrize("kind", ACTS)
def test_activation_values_and_slopes(kind):
    a = np.array([-6.0, -1.5, -0.3, 0.2, 1.0, 4.0])
    f, d = ol.act(a, kind)
    np.testing.assert_allclose(d, diff(lambda t: ol.act(t, kind)[0], a, np.ones_like(a)), atol=1e-8)
    known = {"none": 1.0, "silu": 0.7310585786300049, "gelu": 0.8413447460685429,
             "gelu_tanh": 0.8411919906082768, "relu": 1.0}
    assert abs(f[4] - known[kind]) < 1e-12
    assert ol.act(np.zeros(1), kind)[0][0] == 0.0


def test_rmsnorm_closed_form():
    y, s, rstd = ol.rmsnorm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), eps=0.0)
    assert abs(rstd[0] - 1 / np.sqrt(12.5)) < 1e-15
    np.testing.assert_allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-14)


def test_rmsnorm_backward_is_the_derivative():
    rng = np.random.default_rng(0)
    x, r, w, dy = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=7), \
        rng.normal(size=(3, 7))
    _, s, rstd = ol.rmsnorm(x, w, r, 1e-3, 1.0)
    dx, dw = ol.rmsnorm_backward(dy, s, w, rstd, offset=1.0)
    v, u = rng.normal(size=x.shape), rng.normal(size=7)
    loss = lambda a, b: (ol.rmsnorm(a, b, r, 1e-3, 1.0)[0] * dy).sum()  # noqa: E731
    assert abs(diff(lambda a: loss(a, w), x, v) - (dx * v).sum()) < 1e-7
    assert abs(diff(lambda b: loss(x, b), w, u) - (dw * u).sum()) < 1e-7
    extra = rng.normal(size=x.shape)
    np.testing.assert_allclose(ol.rmsnorm_backward(dy, s, w, rstd, extra, 1.0)[0], dx + extra)


@pytest.mark.parametrize("kind", ACTS)
def test_linear_backward_is_the_derivative(kind):
    rng = np.random.default_rng(1)
    x, W, b = rng.normal(size=(4, 5)), rng.normal(size=(3, 5)), rng.normal(size=3)
    res, dy = rng.normal(size=(4, 3)), rng.normal(size=(4, 3))
    z = ol.linear(x, W, b, res, kind)[1]
    dx, dW, db = ol.products(ol.linear_dz(dy, z, kind), x, W)
    loss = lambda a, w, c: (ol.linear(a, w, c, res, kind)[0] * dy).sum()  # noqa: E731
    for g, f, at in ((dx, lambda t: loss(t, W, b), x), (dW, lambda t: loss(x, t, b), W),
                     (db, lambda t: loss(x, W, t), b)):
        v = rng.normal(size=at.shape)
        assert abs(diff(f, at, v) - (g * v).sum()) < 1e-6


@pytest.mark.parametrize("kind", ACTS[1:])
def test_glu_backward_is_the_derivative(kind):
    rng = np.random.default_rng(2)
    x, W, dy = rng.normal(size=(4, 5)), rng.normal(size=(6, 5)), rng.normal(size=(4, 3))
    z = ol.glu(x, W, kind)[1]
    dx, dW, _ = ol.products(ol.glu_dz(dy, z, kind), x, W)
    loss = lambda a, w: (ol.glu(a, w, kind)[0] * dy).sum()  # noqa: E731
    v, u = rng.normal(size=x.shape), rng.normal(size=W.shape)
    assert abs(diff(lambda t: loss(t, W), x, v) - (dx * v).sum()) < 1e-6
    assert abs(diff(lambda t: loss(x, t), W, u) - (dW * u).sum()) < 1e-6
