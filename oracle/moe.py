"""fp64 oracle of the experts' operators and of the products with a scale per block of
128: numpy, written from the definitions (test infrastructure only)."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def sort(experts: np.ndarray, E: int, align: int):
    """(position [T, k], offsets [E + 1], counts [E]) of the pairs in order."""
    counts = [0] * E
    rank = np.full(experts.shape, -1, np.int64)
    for t, j in np.ndindex(*experts.shape):
        e = int(experts[t, j])
        if 0 <= e < E:
            rank[t, j] = counts[e]
            counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // align) * align)
    position = rank.copy()
    for t, j in np.ndindex(*experts.shape):
        if rank[t, j] >= 0:
            position[t, j] += offsets[int(experts[t, j])]
    return position, np.array(offsets), np.array(counts)


def pairs(position: np.ndarray):
    """(t, j, row) of the pairs that have a row."""
    return [(t, j, int(position[t, j])) for t, j in np.ndindex(*position.shape) if position[t, j] >= 0]


def combine(rows, position, weights=None, residual=None):
    """(y, sum of the terms' magnitudes)."""
    T = position.shape[0]
    y = np.zeros((T, rows.shape[1]))
    size = np.zeros_like(y)
    for t, j, r in pairs(position):
        term = rows[r] * (1.0 if weights is None else weights[t, j])
        y[t] += term
        size[t] += np.abs(term)
    if residual is not None:
        y += residual
        size += np.abs(residual)
    return y, size


def combine_bwd(dy, rows, position, weights):
    """(drows with NaN where no pair has its row, dweights, magnitudes of dweights' terms)."""
    drows = np.full(rows.shape, np.nan)
    dw = np.zeros(position.shape)
    size = np.zeros(position.shape)
    for t, j, r in pairs(position):
        drows[r] = dy[t] * (1.0 if weights is None else weights[t, j])
        dw[t, j] = float(np.dot(dy[t], rows[r]))
        size[t, j] = float(np.dot(np.abs(dy[t]), np.abs(rows[r])))
    return drows, dw, size


def block_maxima(x, down, across):
    """The largest magnitude of each block of down x across of a matrix."""
    R, C = x.shape
    out = np.zeros((-(-R // down), -(-C // across)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.abs(x[i * down:(i + 1) * down, j * across:(j + 1) * across]).max()
    return out


def spread(scale, down, across, shape):
    """The scale of each element."""
    return np.repeat(np.repeat(scale, down, 0), across, 1)[:shape[0], :shape[1]]


def product(x, xs, w, ws, w_rows):
    """(y, sum of the terms' magnitudes) of x W^T: x [T, K] with xs [T, K / 128], w [N, K]
    with ws [N / w_rows, K / 128]."""
    a = x * spread(xs, 1, BLOCK, x.shape)
    b = w * spread(ws, w_rows, BLOCK, w.shape)
    return a @ b.T, np.abs(a) @ np.abs(b).T
