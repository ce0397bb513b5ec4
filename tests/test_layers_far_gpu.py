"""Rows whose offsets pass 2^31 elements: many rows, and few rows far apart.  Products on
small integers equal their 64-bit values; norms stay within the bounds of
tests/layers_parity.py on the first and the last rows."""
import numpy as np
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from oracle import layers as ol
from tests.layers_parity import close, f64
from tests.test_products_exact_gpu import gen, ints, same

pytestmark = pytest.mark.gpu
FAR = 1 << 27  # elements between rows


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def apart(rows, cols, init=None):
    t = torch.empty(rows * FAR, dtype=torch.bfloat16, device="cuda").as_strided((rows, cols), (FAR, 1))
    if init is not None:
        t.copy_(init)
    return t


def blocks(T, step=30000):
    return [slice(i, min(i + step, T)) for i in range(0, T, step)]


def test_many_tokens_and_outputs():
    T, K, N = 270001, 64, 8200
    g = gen(1)
    x, w = ints(g, (T, K)), ints(g, (N, K))
    res = v.linear_fwd(x, w, None, None, act="relu", preact=True)
    w64 = w.double()
    for s in blocks(T):
        z = x[s].double() @ w64.t()
        same(res.preact[s], z)
        same(res.y[s], z.clamp(min=0))
    # z's sign is kept in res.preact; dy: the small integers of z's low bits
    dy = res.y
    for s in blocks(T):
        dy[s] = ((res.preact[s].float() + 1000) % 3 - 1).to(torch.bfloat16)
    got = v.linear_bwd(dy, x, w, res.preact, act="relu", bias_grad=True)
    dw, db = torch.zeros((N, K), dtype=torch.float64, device="cuda"), 0
    for s in blocks(T):
        dz = dy[s].double() * (res.preact[s] > 0)
        same(got.dx[s], dz @ w64)
        dw += dz.t() @ x[s].double()
        db = db + dz.sum(0)
    same(got.dweight, dw)
    same(got.dbias, db)


def test_many_tokens_of_a_gated_layer():
    T, K, n = 140003, 64, 8200
    g = gen(2)
    x, w = ints(g, (T, K), 1), ints(g, (2 * n, K), 1)
    res = v.glu_fwd(x, w, act="relu", preact=True)
    w64 = w.double()
    for s in blocks(T, 10000):
        z = x[s].double() @ w64.t()
        same(res.preact[s], z)
        same(res.y[s], z[:, :n].clamp(min=0) * z[:, n:])


@pytest.mark.parametrize("T", [20, 40])
def test_few_rows_far_apart(T):
    K, N = 264, 520
    g = gen(3)
    x, w, r = apart(T, K, ints(g, (T, K))), ints(g, (N, K)), apart(T, N, ints(g, (T, N), 100))
    y, p = apart(T, N), apart(T, N)
    v.linear_fwd(x, w, None, r, act="relu", preact=p, out=y)
    z = x.double() @ w.double().t()
    same(p, z)
    same(y, z.clamp(min=0) + r.double())
    dy = y
    dy.copy_(ints(g, (T, N)))
    got = v.linear_bwd(dy, x, w, p, act="relu", out=apart(T, K))
    dz = dy.double() * (z > 0)
    same(got.dx, dz @ w.double())
    same(got.dweight, dz.t() @ x.double())


@pytest.mark.parametrize("T,H,far", [(270001, 8200, False), (1100000, 2051, False), (40, 4104, True),
                                     (40, 1001, True)])
def test_norm(T, H, far):
    g = gen(4)

    def rand():
        if far:
            return apart(T, H, torch.randn((T, H), generator=g, device="cuda"))
        return torch.empty((T, H), dtype=torch.bfloat16, device="cuda").normal_(generator=g)

    x, r, w = rand(), rand(), (torch.randn(H, generator=g, device="cuda") * 0.5 + 1).bfloat16()
    y, q = (apart(T, H), apart(T, H)) if far else (None, None)
    a = v.rmsnorm_fwd(x, w, r, out=y, residual_out=q)
    f8 = v.rmsnorm_fwd(x, w, r, fp8=True)
    dy = r  # (its rows are needed no more after the checks below)
    ends = [slice(0, 20)] if far else [slice(0, 64), slice(T - 64, T)]
    e = (H + 32) * 2.0 ** -24
    if far:
        ends.append(slice(T - 20, T))
    for s in ends:
        y64, s64, rstd = ol.rmsnorm(f64(x[s]), f64(w), f64(r[s]), 1e-6)
        close(a.y[s], y64, "bf16", e * np.abs(y64), "y")
        close(a.residual[s], s64, "bf16", 2.0 ** -24 * np.abs(s64), "residual")
        close(a.rstd[s], rstd, "f32", e * rstd, "rstd")
        scale = np.abs(y64).max(axis=1) / 448
        close(f8.scale[s], scale, "f32", e * scale, "scale")
        back = f64(f8.y[s].float()) * f64(f8.scale[s])[:, None]
        assert (np.abs(back - y64) <= np.maximum(np.abs(y64) / 16, scale[:, None] * 2.0 ** -10) * 1.001).all()
    del f8, x
    b = v.rmsnorm_bwd(dy, a.residual, w, a.rstd, out=apart(T, H) if far else None)
    for s in ends:
        d64, s64, rs = f64(dy[s]), f64(a.residual[s]), f64(a.rstd[s])
        dx, _ = ol.rmsnorm_backward(d64, s64, f64(w), rs)
        t, h = np.abs(d64 * f64(w)), np.abs(s64 * rs[:, None])
        close(b.dx[s], dx, "bf16", e * rs[:, None] * (t + h * np.mean(t * h, axis=1, keepdims=True)), "dx")
    dw = torch.zeros(H, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(dw)
    for s in blocks(T, 20000):
        t = dy[s].double() * a.residual[s].double() * a.rstd[s].double()[:, None]
        dw += t.sum(0)
        mag += t.abs().sum(0)
    close(b.dweight, f64(dw), "f32", (T + 32) * 2.0 ** -24 * f64(mag), "dweight")
