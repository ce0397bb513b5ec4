"""GPU parity of the RMS norm with the residual's addition (through the public
binding) against the fp64 oracle; bounds in tests/layers_parity.py.  The fp32
evaluation of y has a relative error of at most (H + 8) 2^-24 from the sum of
squares (halved by the root, all terms positive) and a few roundings: taken as
e = (H + 32) 2^-24 |y|; dx and dw likewise with the magnitudes of their terms."""
import numpy as np
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from oracle import layers as ol
from tests.layers_parity import DT, close, f64, gen, randn
from vocabulary_lm_cross_gb300 import capi

pytestmark = pytest.mark.gpu
E24 = 2.0 ** -24

# one element to rows wider than a CTA's registers; multiples of 16 bytes and odd;
# few rows and enough for the kernels that keep rows in flight
SHAPES = [(1, 1), (3, 8), (1, 4096), (5, 1001), (40, 6656), (2000, 264), (1500, 24), (700, 4100),
          (9, 16392), (7, 40000), (6, 33001), (1300, 2056)]


def make(T, H, dtype, seed, pad=0, wdtype=None):
    g = gen(seed)
    return (randn(g, (T, H), DT[dtype], 1.0, pad), randn(g, (T, H), DT[dtype], 2.0, pad),
            randn(g, (H,), wdtype or DT[dtype], 0.5) + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_and_backward(T, H, dtype):
    x, r, w = make(T, H, dtype, T + H)
    res = v.rmsnorm_fwd(x, w, r, eps=1e-5)
    y, s, rstd = ol.rmsnorm(f64(x), f64(w), f64(r), 1e-5)
    e = (H + 32) * E24
    close(res.y, y, dtype, e * np.abs(y), "y")
    close(res.residual, s, dtype, E24 * np.abs(s), "residual")
    close(res.rstd, rstd, "f32", e * rstd, "rstd")
    assert res.scale is None

    g = gen(T + H + 1)
    dy, dr = randn(g, (T, H), DT[dtype], 0.1), randn(g, (T, H), DT[dtype], 0.1)
    grads = v.rmsnorm_bwd(dy, res.residual, w, res.rstd, dresidual=dr)
    s64, rs64 = f64(res.residual), f64(res.rstd)  # what the call was given
    dx, dw = ol.rmsnorm_backward(f64(dy), s64, f64(w), rs64, f64(dr))
    a, xhat = np.abs(f64(dy) * f64(w)), np.abs(s64 * rs64[:, None])
    terms = rs64[:, None] * (a + xhat * np.mean(a * xhat, axis=1, keepdims=True)) + np.abs(f64(dr))
    close(grads.dx, dx, dtype, e * terms, "dx")
    close(grads.dweight, dw, "f32", (T + 32) * E24 * (np.abs(f64(dy)) * xhat).sum(0), "dweight")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_e4m3_output(T, H, dtype):
    x, r, w = make(T, H, dtype, 3 * T + H)
    res = v.rmsnorm_fwd(x, w, r, fp8=True)
    y, s, _ = ol.rmsnorm(f64(x), f64(w), f64(r), 1e-6)
    scale = np.abs(y).max(axis=1) / 448.0
    e = (H + 32) * E24
    close(res.scale, scale, "f32", e * scale, "scale")
    assert res.y.dtype == torch.float8_e4m3fn
    q = y / scale[:, None]
    # e4m3: 3 mantissa bits, normal above 2^-6, step 2^-9 below
    bound = np.maximum(np.abs(q) * 2.0 ** -4, 2.0 ** -10) * (1 + 1e-5) + e * np.abs(q)
    got = f64(res.y.float())
    assert (np.abs(got - q) <= bound).all()
    assert (np.abs(got).max(axis=1) == 448.0).all()  # the row's largest uses the whole range


def test_no_residual_offset_and_fp32_weight():
    x, _, w = make(33, 1024, "bf16", 5, wdtype=torch.float32)
    res = v.rmsnorm_fwd(x, w, eps=1e-3, weight_offset=1.0)
    assert res.residual is None
    y, s, rstd = ol.rmsnorm(f64(x), f64(w), None, 1e-3, 1.0)
    close(res.y, y, "bf16", 1100 * E24 * np.abs(y), "y")
    dy = randn(gen(6), (33, 1024), DT["bf16"])
    grads = v.rmsnorm_bwd(dy, x, w, res.rstd, weight_offset=1.0)
    dx, dw = ol.rmsnorm_backward(f64(dy), s, f64(w), f64(res.rstd), offset=1.0)
    scale = np.abs(f64(dy) * (f64(w) + 1)).max() * rstd.max() * 4
    close(grads.dx, dx, "bf16", 1100 * E24 * scale, "dx")
    close(grads.dweight, dw, "f32", 65 * E24 * (np.abs(f64(dy)) * np.abs(s * rstd[:, None])).sum(0),
          "dweight")


@pytest.mark.parametrize("T,H", [(17, 264), (1500, 264), (17, 263)])
def test_strided_rows_equal_contiguous_ones_and_padding_is_untouched(T, H):
    x, r, w = make(T, H, "bf16", 8, pad=24)
    xc, rc = x.contiguous(), r.contiguous()
    store = torch.full((T, H + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    a = v.rmsnorm_fwd(x, w, r, out=store[:, :H])
    b = v.rmsnorm_fwd(xc, w, rc)
    assert torch.equal(a.y, b.y) and torch.equal(a.residual, b.residual)
    assert torch.equal(a.rstd, b.rstd) and (store[:, H:] == 7).all()


@pytest.mark.parametrize("T,H", [(7, 512), (1200, 512), (7, 511)])
def test_in_place(T, H):
    x, r, w = make(T, H, "bf16", 9)
    want = v.rmsnorm_fwd(x, w, r)
    for buf, other in ((r.clone(), x), (x.clone(), r)):
        got = v.rmsnorm_fwd(buf if other is r else x, w, buf if other is x else r, residual_out=buf)
        assert torch.equal(got.y, want.y) and torch.equal(buf, want.residual)
    dy, dr = randn(gen(1), (T, H), DT["bf16"]), randn(gen(2), (T, H), DT["bf16"])
    ref = v.rmsnorm_bwd(dy, want.residual, w, want.rstd, dresidual=dr)
    d1 = dy.clone()
    got = v.rmsnorm_bwd(d1, want.residual, w, want.rstd, dresidual=dr, out=d1)
    assert torch.equal(d1, ref.dx) and torch.equal(got.dweight, ref.dweight)
    d2 = dr.clone()
    v.rmsnorm_bwd(dy, want.residual, w, want.rstd, dresidual=d2, out=d2)
    assert torch.equal(d2, ref.dx)


def test_accumulated_weight_gradient():
    x, r, w = make(50, 96, "f32", 10)
    res = v.rmsnorm_fwd(x, w, r)
    dy = randn(gen(3), (50, 96), torch.float32)
    one = v.rmsnorm_bwd(dy, res.residual, w, res.rstd).dweight
    acc = one.clone()
    v.rmsnorm_bwd(dy, res.residual, w, res.rstd, dweight=acc, accumulate_dweight=True)
    assert torch.equal(acc, one + one)


def test_no_rows():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    res = v.rmsnorm_fwd(x, w, x)
    assert res.y.shape == (0, 64) and res.rstd.shape == (0,)
    dw = torch.full((64,), 3.0, device="cuda")
    assert (v.rmsnorm_bwd(x, x, w, res.rstd, dweight=dw, accumulate_dweight=True).dweight == 3).all()
    assert (v.rmsnorm_bwd(x, x, w, res.rstd, dweight=dw).dweight == 0).all()


def test_rows_of_zeros_and_non_finite_values_stay_in_their_row():
    x, r, w = make(6, 264, "bf16", 11)
    x[1], r[1] = 0, 0
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    res, q = v.rmsnorm_fwd(x, w, r), v.rmsnorm_fwd(x, w, r, fp8=True)
    y = ol.rmsnorm(f64(x[[0, 2, 5]]), f64(w), f64(r[[0, 2, 5]]), 1e-6)[0]
    close(res.y[[0, 2, 5]], y, "bf16", 300 * E24 * np.abs(y), "y")
    assert (res.y[1] == 0).all() and abs(float(res.rstd[1]) - 1000.0) < 1e-3
    assert (q.y[1].float() == 0).all() and torch.isfinite(q.scale[[0, 1, 2, 5]]).all()
    assert torch.isnan(res.y[3]).all() and torch.isnan(q.scale[3])
    assert torch.isnan(res.y[4, 7]) and float(res.rstd[4]) == 0.0


def test_weight_gradient_matches_differences():
    x, r, w = make(20, 264, "f32", 12)
    dy = randn(gen(4), (20, 264), torch.float32)
    res = v.rmsnorm_fwd(x, w, r)
    grads = v.rmsnorm_bwd(dy, res.residual, w, res.rstd)
    rng = np.random.default_rng(0)
    for g, at, f in ((grads.dx, f64(x), lambda t: ol.rmsnorm(t, f64(w), f64(r))[0]),
                     (grads.dweight, f64(w), lambda t: ol.rmsnorm(f64(x), t, f64(r))[0])):
        d = rng.normal(size=at.shape)
        h = 1e-4
        slope = ((f(at + h * d) - f(at - h * d)) * f64(dy)).sum() / (2 * h)
        assert abs(slope - (f64(g) * d).sum()) <= 1e-5 * (np.abs(f64(g) * d).sum() + 1)


def test_repeated_calls_on_another_stream_give_the_same_bits():
    x, r, w = make(1400, 1032, "bf16", 13)
    dy = randn(gen(5), (1400, 1032), DT["bf16"])
    a = v.rmsnorm_fwd(x, w, r)
    b = v.rmsnorm_bwd(dy, a.residual, w, a.rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            c = v.rmsnorm_fwd(x, w, r)
            d = v.rmsnorm_bwd(dy, c.residual, w, c.rstd)
    s.synchronize()
    assert torch.equal(a.y, c.y) and torch.equal(b.dx, d.dx) and torch.equal(b.dweight, d.dweight)


def test_binding_refuses():
    x, r, w = make(4, 64, "bf16", 14)
    with pytest.raises(TypeError):
        v.rmsnorm_fwd(x.to(torch.float8_e4m3fn), w)
    with pytest.raises(TypeError):
        v.rmsnorm_fwd(x.cpu(), w)
    with pytest.raises(ValueError):
        v.rmsnorm_fwd(x, w[:32])
    with pytest.raises(ValueError):
        v.rmsnorm_fwd(x, w, r[:2])
    with pytest.raises(ValueError):
        v.rmsnorm_fwd(x.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        v.rmsnorm_fwd(x, w, residual_out=r)
    with pytest.raises(capi.VlmceError):
        v.rmsnorm_fwd(x, w, r, out=x)
    rstd = v.rmsnorm_fwd(x, w).rstd
    with pytest.raises(TypeError):
        v.rmsnorm_bwd(x.float(), x, w, rstd)
    with pytest.raises(ValueError):
        v.rmsnorm_bwd(x, x, w, rstd, accumulate_dweight=True)
    with pytest.raises(capi.VlmceError):
        v.rmsnorm_bwd(r, x, w, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("T,H", [(1, 40), (333, 1001), (512, 264), (512, 4100), (513, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weight_gradient_added_to_and_in_place(T, H, dtype):
    x, r, w = make(T, H, dtype, 21)
    res = v.rmsnorm_fwd(x, w, r)
    dy = randn(gen(22), (T, H), DT[dtype])
    a = v.rmsnorm_bwd(dy, res.residual, w, res.rstd)
    acc = a.dweight.clone()
    v.rmsnorm_bwd(dy, res.residual, w, res.rstd, dweight=acc, accumulate_dweight=True)
    d = dy.clone()
    b = v.rmsnorm_bwd(d, res.residual, w, res.rstd, out=d)
    s64, rs64 = f64(res.residual), f64(res.rstd)
    dw = ol.rmsnorm_backward(f64(dy), s64, f64(w), rs64)[1]
    e = (T + 32) * E24 * (np.abs(f64(dy)) * np.abs(s64 * rs64[:, None])).sum(0)
    close(a.dweight, dw, "f32", e, "dweight")
    assert torch.equal(acc, a.dweight + a.dweight)
    assert torch.equal(a.dx, d) and torch.equal(a.dweight, b.dweight)


# rows that start at any alignment, enough of them for the kernels that keep rows in
# flight; pad: elements between rows (every stride of a case has the same remainder)
SHIFTED = [(4000, 1, 0), (4001, 9, 0), (3700, 501, 0), (3651, 263, 24), (1300, 2051, 8),
           (2000, 1002, 6), (950, 4085, 0), (2000, 1004, 4), (1250, 3333, 0), (920, 8185, 0)]


def strided(t, pad):
    store = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    store[:, :t.shape[1]] = t
    return store, store[:, :t.shape[1]]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,pad", SHIFTED)
def test_rows_at_any_alignment(T, H, pad, dtype):
    x, r, w = make(T, H, dtype, 7 * T + H)
    e = (H + 32) * E24
    y, s, rstd = ol.rmsnorm(f64(x), f64(w), f64(r), 1e-5)
    (xs, xv), (rs, rv) = strided(x, pad), strided(r, pad)
    (ys, yv), (ss, sv) = strided(torch.zeros_like(x), pad), strided(torch.zeros_like(x), pad)
    res = v.rmsnorm_fwd(xv, w, rv, eps=1e-5, out=yv, residual_out=sv)
    close(yv, y, dtype, e * np.abs(y), "y")
    close(sv, s, dtype, E24 * np.abs(s), "residual")
    close(res.rstd, rstd, "f32", e * rstd, "rstd")
    assert torch.isnan(ys[:, H:]).all() and torch.isnan(ss[:, H:]).all()

    q8 = v.rmsnorm_fwd(x, w, r, eps=1e-5, fp8=True)
    scale = rstd * np.maximum(np.abs(s * f64(w)).max(axis=1), 1e-30) / 448.0
    close(q8.scale, scale, "f32", e * scale, "scale")
    q = y / scale[:, None]
    bound = np.maximum(np.abs(q) * 2.0 ** -4, 2.0 ** -10) * (1 + 1e-5) + e * np.abs(q)
    assert (np.abs(f64(q8.y.float()) - q) <= bound).all()
    close(q8.residual, s, dtype, E24 * np.abs(s), "residual")

    g = gen(T + H + 1)
    dy, dr = randn(g, (T, H), DT[dtype], 0.1), randn(g, (T, H), DT[dtype], 0.1)
    (_, dyv), (_, drv), (dxs, dxv) = strided(dy, pad), strided(dr, pad), strided(dy, pad)
    grads = v.rmsnorm_bwd(dyv, sv, w, res.rstd, dresidual=drv, out=dxv)
    s64, rs64 = f64(sv), f64(res.rstd)
    dx, dw = ol.rmsnorm_backward(f64(dy), s64, f64(w), rs64, f64(dr))
    a, xhat = np.abs(f64(dy) * f64(w)), np.abs(s64 * rs64[:, None])
    terms = rs64[:, None] * (a + xhat * np.mean(a * xhat, axis=1, keepdims=True)) + np.abs(f64(dr))
    close(dxv, dx, dtype, e * terms, "dx")
    close(grads.dweight, dw, "f32", (T + 32) * E24 * (np.abs(f64(dy)) * xhat).sum(0), "dweight")
    assert torch.isnan(dxs[:, H:]).all()
    # over dy, and over dresidual
    for buf in (dyv, drv):
        got = v.rmsnorm_bwd(dyv, sv, w, res.rstd, dresidual=drv, out=buf)
        assert torch.equal(buf, dxv) and torch.equal(got.dweight, grads.dweight)
        buf.copy_(dy if buf is dyv else dr)
    # the sum over x
    got = v.rmsnorm_fwd(xv, w, rv, eps=1e-5, out=yv, residual_out=xv)
    assert torch.equal(xv, sv) and torch.equal(got.rstd, res.rstd)


@pytest.mark.parametrize("wdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(4000, 501), (1000, 4085)])
def test_rows_at_any_alignment_keep_non_finite_values_to_themselves(T, H, wdtype):
    x, r, w = make(T, H, "bf16", 31, wdtype=wdtype)
    clean = v.rmsnorm_fwd(x, w, r, weight_offset=1.0)
    dy = randn(gen(32), (T, H), DT["bf16"])
    ref = v.rmsnorm_bwd(dy, clean.residual, w, clean.rstd, weight_offset=1.0)
    bad = torch.arange(1, T, 3, device="cuda")
    x2, dy2 = x.clone(), dy.clone()
    x2[bad] = float("nan")
    x2[bad[::2]] = float("inf")
    dy2[bad] = float("nan")
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[bad] = False
    got = v.rmsnorm_fwd(x2, w, r, weight_offset=1.0)
    assert torch.equal(got.y[good], clean.y[good])
    assert torch.equal(got.residual[good], clean.residual[good])
    assert not torch.isfinite(got.y[bad]).all(dim=1).any()
    grads = v.rmsnorm_bwd(dy2, clean.residual, w, clean.rstd, weight_offset=1.0)
    assert torch.equal(grads.dx[good], ref.dx[good]) and torch.isnan(grads.dx[bad]).all()
