"""fp64 oracle of the decoder-layer operators (test infrastructure): the RMS norm
with the residual's addition, the linear layer (bias, activation, residual) and
the gated layer, forward and backward, from their definitions in plain numpy.

    s = x + residual, rstd = (mean_j s_j^2 + eps)^-1/2, y = s rstd (w + offset)
    z = x W^T + b, y = act(z) + residual
    (g | u) = x W^T, y = act(g) u

Backward functions return the gradients for an upstream gradient dy.
"""
from __future__ import annotations

import math

import numpy as np

C0, C1 = math.sqrt(2.0 / math.pi), 0.044715
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def _sigmoid(a):
    e = np.exp(-np.abs(a))
    return np.where(a >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(a: np.ndarray, kind: str):
    """(act(a), act'(a))."""
    a = np.asarray(a, np.float64)
    if kind == "none":
        return a, np.ones_like(a)
    if kind == "relu":
        return np.where(a > 0, a, 0.0), np.where(a > 0, 1.0, 0.0)
    if kind == "silu":
        s = _sigmoid(a)
        return a * s, s * (1.0 + a * (1.0 - s))
    if kind == "gelu":
        p = 0.5 * _erfc(-a / math.sqrt(2.0)).reshape(a.shape)
        return a * p, p + a * np.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        t = np.tanh(C0 * (a + C1 * a ** 3))
        return (0.5 * a * (1.0 + t),
                0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * C0 * (1.0 + 3.0 * C1 * a * a))
    raise ValueError(kind)


def rmsnorm(x, w, residual=None, eps=1e-6, offset=0.0):
    """(y, s, rstd)."""
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s * rstd[:, None] * (w + offset), s, rstd


def rmsnorm_backward(dy, s, w, rstd, dresidual=None, offset=0.0):
    """(dx, dw)."""
    xhat = s * rstd[:, None]
    a = dy * (w + offset)
    dx = rstd[:, None] * (a - xhat * np.mean(a * xhat, axis=1, keepdims=True))
    return dx if dresidual is None else dx + dresidual, np.sum(dy * xhat, axis=0)


def linear(x, W, bias=None, residual=None, kind="none"):
    """(y, z)."""
    z = x @ W.T
    if bias is not None:
        z = z + bias
    y = act(z, kind)[0]
    return (y if residual is None else y + residual), z


def linear_dz(dy, z, kind):
    return dy if kind == "none" else dy * act(z, kind)[1]


def glu(x, W, kind="silu"):
    """(y, z) with z = (g | u)."""
    z = x @ W.T
    n = W.shape[0] // 2
    return act(z[:, :n], kind)[0] * z[:, n:], z


def glu_dz(dy, z, kind):
    n = z.shape[1] // 2
    f, d = act(z[:, :n], kind)
    return np.concatenate([dy * z[:, n:] * d, dy * f], axis=1)


def products(dz, x, W):
    """(dx, dW, db) from the gradient of the pre-activations."""
    return dz @ W, dz.T @ x, dz.sum(axis=0)
