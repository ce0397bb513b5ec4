"""GPU parity of the linear and gated layers (through the public binding) against
the fp64 oracle; elementwise bounds from tests/layers_parity.py."""
import numpy as np
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from oracle import layers as ol
from tests.layers_parity import DT, E23, TINY, U16, close, f64, gen, randn
from vocabulary_lm_cross_gb300 import capi

pytestmark = pytest.mark.gpu
ACTS = ["none", "silu", "gelu", "gelu_tanh", "relu"]

# (T, K, N): one token; tokens and outputs around the tiles' 16, 128 and 256; one
# weight row; K of one chunk and of none whole; sizes for K split over a cluster,
# several token tiles, and pair tiles with a ragged edge
SHAPES = [(1, 8, 1), (1, 4096, 384), (2, 72, 129), (17, 1000, 127), (64, 2048, 256), (130, 520, 300),
          (257, 264, 77), (300, 640, 1031), (1025, 1032, 520), (2100, 136, 2056)]


def fp32_bound(x, W, K):
    return (K + 8) * E23 * (np.abs(x) @ np.abs(W).T)


def linear_case(T, K, N, dtype, seed, gated=False, pad=0):
    g = gen(seed)
    x = randn(g, (T, K), DT[dtype], 1.0, pad)
    w = randn(g, ((2 if gated else 1) * N, K), DT[dtype], K ** -0.5, pad)
    return g, x, w


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("kind", ACTS)
def test_linear_forward_and_backward(T, K, N, dtype, kind):
    g, x, w = linear_case(T, K, N, dtype, T + K + N)
    b, r = randn(g, (N,), DT[dtype]), randn(g, (T, N), DT[dtype])
    res = v.linear_fwd(x, w, b, r, act=kind, preact=True)
    x64, w64 = f64(x), f64(w)
    y, z = ol.linear(x64, w64, f64(b), f64(r), kind)
    e = fp32_bound(x64, w64, K) + E23 * np.abs(z)
    close(res.preact, z, dtype, e, "preact")
    close(res.y, y, dtype, 1.2 * e + 3e-6 * (1 + np.abs(z)) + E23 * np.abs(y), "y")

    dy = randn(g, (T, N), DT[dtype], 0.5)
    for wdt in (torch.float32, DT[dtype]):
        grads = v.linear_bwd(dy, x, w, res.preact, act=kind, bias_grad=True, dweight_dtype=wdt)
        check_grads(grads, ol.linear_dz(f64(dy), f64(res.preact), kind), x64, w64, dtype, kind,
                    np.abs(f64(dy)))


def check_grads(grads, dz, x64, w64, dtype, kind, scale):
    """scale: bounds |d dz / d act'|, for the error of the slopes."""
    (T, R), K = dz.shape, x64.shape[1]
    e_dz = 4e-6 * (np.abs(dz) + scale)                # the activation's fp32 evaluation
    if kind != "none":
        e_dz = e_dz + U16[dtype] * np.abs(dz) + TINY[dtype] / 2  # dz in 16 bits
    else:
        e_dz = 0 * dz
    adz = np.abs(dz)
    dx, dw, db = ol.products(dz, x64, w64)
    close(grads.dx, dx, dtype, e_dz @ np.abs(w64) + (R + 8) * E23 * (adz @ np.abs(w64)), "dx")
    wide = "f32" if grads.dweight.dtype == torch.float32 else dtype
    close(grads.dweight, dw, wide, e_dz.T @ np.abs(x64) + (T + 8) * E23 * (adz.T @ np.abs(x64)),
          "dweight")
    if grads.dbias is not None:
        slopes = 4e-6 * (adz + scale) if kind != "none" else 0 * adz
        close(grads.dbias, db, "f32", slopes.sum(0) + (T + 8) * E23 * adz.sum(0), "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("kind", ACTS[1:])
def test_glu_forward_and_backward(T, K, N, dtype, kind):
    g, x, w = linear_case(T, K, N, dtype, 2 * T + K + N, gated=True)
    res = v.glu_fwd(x, w, act=kind, preact=True)
    x64, w64 = f64(x), f64(w)
    y, z = ol.glu(x64, w64, kind)
    e = fp32_bound(x64, w64, K)
    close(res.preact, z, dtype, e, "preact")
    a, u = np.abs(ol.act(z[:, :N], kind)[0]), np.abs(z[:, N:])
    e_a = 1.2 * e[:, :N] + 3e-6 * (1 + np.abs(z[:, :N]))
    close(res.y, y, dtype, e_a * (u + e[:, N:]) + a * e[:, N:] + E23 * np.abs(y), "y")
    assert torch.equal(v.glu_fwd(x, w, act=kind).y, res.y)

    dy = randn(g, (T, N), DT[dtype], 0.5)
    z64 = f64(res.preact)
    scale = np.abs(f64(dy)) * (1 + np.maximum(np.abs(z64[:, :N]), np.abs(z64[:, N:])))
    for wdt in (torch.float32, DT[dtype]):
        grads = v.glu_bwd(dy, x, w, res.preact, act=kind, dweight_dtype=wdt)
        assert grads.dbias is None
        check_grads(grads, ol.glu_dz(f64(dy), z64, kind), x64, w64, dtype, kind,
                    np.concatenate([scale, scale], axis=1))


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T,K,N", [(1, 16, 1), (1, 4096, 384), (17, 1008, 127), (64, 4096, 256),
                                   (300, 640, 1031), (1025, 1040, 520), (2100, 144, 2056)])
def test_e4m3_operands(T, K, N, gated, out):
    g = gen(T + K)
    rows = (2 if gated else 1) * N
    x = randn(g, (T, K), torch.float32, 20.0).to(torch.float8_e4m3fn)
    w = randn(g, (rows, K), torch.float32, 20.0).to(torch.float8_e4m3fn)
    xs = (torch.rand(T, generator=g) * 0.1 + 0.01).cuda()
    ws = (torch.rand(rows, generator=g) * 0.01 / K ** 0.5 + 1e-4).cuda()
    x64 = f64(x.float()) * f64(xs)[:, None]
    w64 = f64(w.float()) * f64(ws)[:, None]
    e = fp32_bound(x64, w64, K)
    kw = dict(x_scale=xs, weight_scale=ws, out_dtype=DT[out])
    if gated:
        res = v.glu_fwd(x, w, preact=True, **kw)
        y, z = ol.glu(x64, w64)
        e_a = 1.2 * e[:, :N] + 3e-6 * (1 + np.abs(z[:, :N]))
        e_y = e_a * (np.abs(z[:, N:]) + e[:, N:]) + np.abs(z[:, :N]) * e[:, N:]
        close(res.preact, z, out, e + 3 * E23 * np.abs(z), "preact")
        close(res.y, y, out, e_y + 4 * E23 * np.abs(y), "y")
    else:
        b, r = randn(g, (N,), DT[out]), randn(g, (T, N), DT[out])
        res = v.linear_fwd(x, w, b, r, act="silu", **kw)
        y, z = ol.linear(x64, w64, f64(b), f64(r), "silu")
        close(res.y, y, out, 1.2 * (e + 4 * E23 * np.abs(z)) + 3e-6 * (1 + np.abs(z)) +
              E23 * np.abs(y), "y")


@pytest.mark.parametrize("T", [1, 40, 700, 2100])
def test_strides_and_in_place_residual(T):
    K, N = 264, 1040
    g, x, w = linear_case(T, K, N, "bf16", 7, pad=8)
    r = randn(g, (T, N), DT["bf16"])
    want = v.linear_fwd(x.contiguous(), w.contiguous(), None, r).y
    store = torch.full((T, N + 3), 5.0, dtype=torch.bfloat16, device="cuda")  # odd stride
    assert torch.equal(v.linear_fwd(x, w, None, r, out=store[:, :N]).y, want)
    assert (store[:, N:] == 5).all()
    wide = torch.full((T, N + 8), 5.0, dtype=torch.bfloat16, device="cuda")[:, :N]
    wide.copy_(r)
    v.linear_fwd(x, w, None, wide, out=wide)
    assert torch.equal(wide, want)
    odd = store[:, :N]
    odd.copy_(r)
    v.linear_fwd(x, w, None, odd, out=odd)
    assert torch.equal(odd, want) and (store[:, N:] == 5).all()
    # gradients of strided operands
    dy = randn(g, (T, N), DT["bf16"], 1.0, pad=5)
    a = v.linear_bwd(dy, x, w, bias_grad=True)
    b = v.linear_bwd(dy.contiguous(), x.contiguous(), w.contiguous(), bias_grad=True)
    for i in range(3):
        assert torch.equal(a[i], b[i])


def test_accumulation_and_parts():
    T, K, N = 100, 128, 72
    g, x, w = linear_case(T, K, N, "bf16", 8)
    dy = randn(g, (T, N), DT["bf16"])
    full = v.linear_bwd(dy, x, w, bias_grad=True)
    dw, db = full.dweight.clone(), full.dbias.clone()
    got = v.linear_bwd(dy, x, w, dweight=dw, dbias=db, accumulate=True, want_dx=False)
    assert got.dx is None and got.dweight is dw
    assert torch.equal(dw, full.dweight + full.dweight) and torch.equal(db, full.dbias + full.dbias)
    only = v.linear_bwd(dy, x, w, want_dweight=False)
    assert torch.equal(only.dx, full.dx) and only.dweight is None and only.dbias is None


def test_no_tokens():
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    dy = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert v.linear_fwd(x, w).y.shape == (0, 32)
    assert v.glu_fwd(x, w).y.shape == (0, 16)
    dw, db = torch.ones((32, 64), device="cuda"), torch.ones(32, device="cuda")
    v.linear_bwd(dy, x, w, dweight=dw, dbias=db, accumulate=True)
    assert (dw == 1).all() and (db == 1).all()
    v.linear_bwd(dy, x, w, dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("T", [3, 400, 2100])
def test_non_finite_values_stay_with_their_token_and_output(T):
    K, N = 264, 520
    g, x, w = linear_case(T, K, N, "bf16", 9)
    clean = v.linear_fwd(x, w, act="relu").y.clone()
    x[1, 3] = float("nan")
    w[5, 0] = float("inf")
    y = v.linear_fwd(x, w, act="relu").y
    assert torch.isnan(y[1]).all()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[1] = False
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[5] = False
    assert torch.equal(y[keep][:, cols], clean[keep][:, cols])
    assert not torch.isfinite(y[keep][:, 5]).all()


def test_large_pre_activations_have_finite_slopes():
    z = torch.tensor([[-3e38, -1e5, -30.0, 0.0, 30.0, 1e5, 3e38, 1.0]], device="cuda").bfloat16()
    dy = torch.ones((1, 8), device="cuda").bfloat16()
    eye = torch.eye(8, device="cuda").bfloat16()
    for kind in ACTS[1:]:
        d = v.linear_bwd(dy, eye[:1], eye, z, act=kind).dx.float()[0]
        want = ol.act(f64(z)[0].clip(-700, 700), kind)[1]
        assert np.abs(f64(d) - want).max() < 0.01, kind


@pytest.mark.parametrize("gated", [False, True])
def test_gradients_match_differences(gated):
    T, K, N = 24, 64, 40
    g, x, w = linear_case(T, K, N, "f16", 10, gated)
    dy = randn(g, (T, N), DT["f16"])
    fwd, bwd = (v.glu_fwd, v.glu_bwd) if gated else (v.linear_fwd, v.linear_bwd)
    ref = ol.glu if gated else lambda a, b, k: ol.linear(a, b, kind=k)
    z = fwd(x, w, act="gelu", preact=True).preact
    grads = bwd(dy, x, w, z, act="gelu", dweight_dtype=torch.float32)
    x64, w64, rng, h = f64(x), f64(w), np.random.default_rng(0), 1e-4
    for got, at, f in ((grads.dx, x64, lambda t: ref(t, w64, "gelu")[0]),
                       (grads.dweight, w64, lambda t: ref(x64, t, "gelu")[0])):
        d = rng.normal(size=at.shape)
        slope = ((f(at + h * d) - f(at - h * d)) * f64(dy)).sum() / (2 * h)
        # z, dz and dx in fp16: 2^-11 each, at most
        assert abs(slope - (f64(got) * d).sum()) <= 2 * 2.0 ** -11 * np.abs(f64(got) * d).sum()


@pytest.mark.parametrize("T", [1, 300, 1500])
def test_calls_in_a_row_on_another_stream_and_in_a_graph_give_the_same_bits(T):
    K, N = 512, 1040
    g, x, w = linear_case(T, K, N, "bf16", 11, gated=True)
    dy = randn(g, (T, N), DT["bf16"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        f = v.glu_fwd(x, w, preact=True, dev_err=err)
        b = v.glu_bwd(dy, x, w, f.preact, dev_err=err)
        return f.y, f.preact, b.dx, b.dweight

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            got = step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            captured = step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, captured):
        assert torch.equal(a, b) and torch.equal(a, c)
    assert int(err) == 0


def test_binding_refuses():
    g, x, w = linear_case(4, 64, 32, "bf16", 12)
    dy = randn(g, (4, 32), DT["bf16"])
    with pytest.raises(TypeError):
        v.linear_fwd(x.float(), w.float())
    with pytest.raises(TypeError):
        v.linear_fwd(x, w.half())
    with pytest.raises(TypeError):
        v.linear_fwd(x.cpu(), w)
    with pytest.raises(ValueError):
        v.linear_fwd(x, w[:, :32])
    with pytest.raises(ValueError):
        v.linear_fwd(x, w, act="tanh")
    with pytest.raises(ValueError):
        v.glu_fwd(x, w, act="none")
    with pytest.raises(ValueError):
        v.glu_fwd(x, w[:31])
    with pytest.raises(ValueError):
        v.linear_fwd(x, w, x_scale=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        v.linear_fwd(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn))
    with pytest.raises(TypeError):
        v.linear_fwd(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        v.linear_fwd(x, w, dy[0, :16])
    with pytest.raises(capi.VlmceError):
        v.linear_fwd(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(ValueError):
        v.linear_bwd(dy, x, w, act="silu")
    with pytest.raises(ValueError):
        v.linear_bwd(dy, x, w, accumulate=True)
    with pytest.raises(capi.VlmceError):
        v.linear_bwd(dy, x, w, dweight=torch.zeros((32, 64), device="cuda").bfloat16(),
                     accumulate=True)
    with pytest.raises(TypeError):
        v.linear_bwd(dy.to(torch.float8_e4m3fn), x.to(torch.float8_e4m3fn),
                     w.to(torch.float8_e4m3fn))
    with pytest.raises(capi.VlmceError):
        v.linear_bwd(dy, x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_workspace_may_be_missing_where_dy_is_read_as_it_is():
    T, K, N = 40, 64, 72
    g, x, w = linear_case(T, K, N, "bf16", 30)
    dy, z = randn(g, (T, N), DT["bf16"]), randn(g, (T, N), DT["bf16"])
    lib, s = capi.lib(), torch.cuda.current_stream().cuda_stream
    dx, db = torch.empty_like(x), torch.empty(N, device="cuda")

    def call(act, db_ptr, ws):
        return lib.linear_bwd(dy.data_ptr(), N, x.data_ptr(), K, w.data_ptr(), K, z.data_ptr(), N,
                              capi.BF16, T, N, K, act, dx.data_ptr(), K, None, capi.F32, db_ptr, 0,
                              None, ws.data_ptr() if ws is not None else None,
                              ws.numel() if ws is not None else 0, s)

    assert call(capi.ACT_NONE, None, None) == capi.OK
    full = torch.empty(lib.vlmce_linear_bwd_workspace_bytes(T, N, K), dtype=torch.uint8,
                       device="cuda")
    got = dx.clone()
    assert call(capi.ACT_NONE, None, full) == capi.OK
    assert torch.equal(got, dx)
    assert call(capi.ACT_NONE, db.data_ptr(), None) == capi.ERR_WORKSPACE_TOO_SMALL
    assert call(capi.ACT_SILU, None, None) == capi.ERR_WORKSPACE_TOO_SMALL
    assert call(capi.ACT_NONE, None, full[:256]) == capi.ERR_WORKSPACE_TOO_SMALL


def placed(t, pad, offset):
    """t's rows `pad` elements apart from `offset` elements on, NaN around them."""
    rows, cols = t.shape
    store = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), dtype=t.dtype,
                       device=t.device)
    v_ = store.as_strided((rows, cols), (cols + pad, 1), offset)
    v_.copy_(t)
    return v_


# columns around a thread's 8 and a block's 256; (pad, offset) of dy and of preact
@pytest.mark.parametrize("N", [1, 2, 5, 7, 8, 9, 12, 255, 256, 257, 263, 511, 1031])
@pytest.mark.parametrize("T,places", [(1, ((0, 1), (0, 0))), (9, ((0, 0), (0, 3))), (70, ((1, 2), (2, 5))),
                                      (300, ((3, 7), (0, 0)))])
def test_gradients_of_rows_at_any_alignment(T, N, places):
    K = 40
    for gated, kind in ((False, "none"), (False, "gelu"), (True, "silu")):
        g, x, w = linear_case(T, K, N, "bf16", T + N, gated)
        pre = None if kind == "none" else placed(randn(g, (T, 2 * N if gated else N), DT["bf16"]),
                                                 *places[1])
        dy = placed(randn(g, (T, N), DT["bf16"], 0.5), *places[0])
        z64 = None if pre is None else f64(pre)
        if gated:
            grads = v.glu_bwd(dy, x, w, pre, act=kind, dweight_dtype=torch.float32)
            dz = ol.glu_dz(f64(dy), z64, kind)
            scale = np.concatenate([np.abs(f64(dy) * z64[:, N:]), np.abs(f64(dy))], axis=1)
        else:
            grads = v.linear_bwd(dy, x, w, pre, act=kind, bias_grad=True, dweight_dtype=torch.float32)
            dz = f64(dy) if kind == "none" else ol.linear_dz(f64(dy), z64, kind)
            scale = np.abs(f64(dy))
        check_grads(grads, dz, f64(x), f64(w), "bf16", kind, scale)


@pytest.mark.parametrize("N,pad,offset", [(1031, 0, 0), (1032, 1, 3), (1033, 3, 7), (1030, 2, 2), (1029, 0, 5),
                                          (257, 6, 1), (65, 0, 1)])
def test_residual_at_any_alignment(N, pad, offset):
    T, K = 2100, 72
    g, x, w = linear_case(T, K, N, "bf16", N)
    b, r = randn(g, (N,), DT["bf16"]), placed(randn(g, (T, N), DT["bf16"]), pad, offset)
    y, z = ol.linear(f64(x), f64(w), f64(b), f64(r), "silu")
    e = fp32_bound(f64(x), f64(w), K) + E23 * np.abs(z)
    bound = 1.2 * e + 3e-6 * (1 + np.abs(z)) + E23 * np.abs(y)
    for out in (torch.empty_like(y_ := torch.empty((T, N), dtype=DT["bf16"], device="cuda")),
                placed(y_, pad, offset), placed(y_, -N % 8, 0), r):
        res = v.linear_fwd(x, w, b, r, act="silu", out=out)
        close(res.y, y, "bf16", bound, "y")
