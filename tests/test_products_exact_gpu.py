"""Products of the linear and gated layers on small integers: every product and partial
sum is an integer below 2^24, so fp32 accumulation is exact in any order and the results
equal a plain 64-bit evaluation, rounded once, bit for bit.  A missing, doubled or
misplaced element of K, or a tile handed out wrongly, shows at any size."""
import pytest
import torch

import vocabulary_lm_cross_gb300 as v

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def ints(g, shape, most=2, dtype="bf16"):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(torch.float32).to(DT[dtype])


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def same(got, want64):
    """got equals want64 rounded once to its type."""
    assert float(want64.abs().max()) < 2 ** 24
    want = want64.to(got.dtype)
    assert torch.equal(got, want), (int((got != want).sum()), (got != want).nonzero()[0].tolist())


def scales(g, n):
    """Powers of two: products with them are exact."""
    return torch.exp2(torch.randint(-2, 2, (n,), generator=g, device="cuda").float())


def check_linear_fwd(T, K, N, dtype, seed=0, residual=True, in_place=False):
    g = gen(seed)
    x, w = ints(g, (T, K), dtype=dtype), ints(g, (N, K), dtype=dtype)
    z = x.double() @ w.double().t()
    odt = "bf16" if dtype == "e4m3" else dtype
    kw = {}
    if dtype == "e4m3":
        kw = dict(x_scale=scales(g, T), weight_scale=scales(g, N))
        z = z * kw["x_scale"].double()[:, None] * kw["weight_scale"].double()
    b = ints(g, (N,), 100, odt)
    r = ints(g, (T, N), 100, odt) if residual else None
    z = z + b.double()
    y = z.clamp(min=0)
    if residual:
        y = y + r.double()
    res = v.linear_fwd(x, w, b, r, act="relu", preact=True, out=r if in_place else None, **kw)
    same(res.preact, z)
    same(res.y, y)


def check_glu_fwd(T, K, n, dtype, seed=0, out_dtype=None):
    g = gen(seed)
    x, w = ints(g, (T, K), 1, dtype), ints(g, (2 * n, K), 1, dtype)
    z = x.double() @ w.double().t()
    kw = {}
    if dtype == "e4m3":
        kw = dict(x_scale=scales(g, T), weight_scale=scales(g, 2 * n))
        z = z * kw["x_scale"].double()[:, None] * kw["weight_scale"].double()
    res = v.glu_fwd(x, w, act="relu", preact=True, **kw)
    same(res.preact, z)
    same(res.y, z[:, :n].clamp(min=0) * z[:, n:])


def check_bwd(T, K, N, dtype="bf16", seed=0, gated=False, wide=True, accumulate=False):
    """dx and dweight; relu and small integers keep dz exact in 16 bits."""
    g = gen(seed)
    R = 2 * N if gated else N
    x, w, dy, z = ints(g, (T, K), dtype=dtype), ints(g, (R, K), dtype=dtype), \
        ints(g, (T, N), dtype=dtype), ints(g, (T, R), dtype=dtype)
    z64, dy64 = z.double(), dy.double()
    on = (z64[:, :N] > 0).double()
    dz = torch.cat([dy64 * z64[:, N:] * on, dy64 * z64[:, :N] * on], 1) if gated else dy64 * on
    dw = dz.t() @ x.double()
    kw = dict(dweight_dtype=torch.float32 if wide else DT[dtype])
    if accumulate:
        start = ints(g, (R, K), 1000).float()
        dw = dw + start.double()
        kw = dict(dweight=start, accumulate=True)
    got = (v.glu_bwd if gated else v.linear_bwd)(dy, x, w, z, act="relu", **kw)
    same(got.dx, dz @ w.double())
    same(got.dweight, dw)


# pairs that take several tiles each by cluster launch control (K of 32 chunks and more)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pairs_that_ask_for_their_next_tile_forward(dtype):
    for seed in range(3):
        check_linear_fwd(4352, 2056, 2600, dtype, seed)
    check_glu_fwd(4400, 2120, 1330, dtype)


def test_pairs_that_ask_for_their_next_tile_e4m3():
    check_linear_fwd(4352, 4112, 2600, "e4m3")
    check_glu_fwd(4400, 4240, 1330, "e4m3")


@pytest.mark.parametrize("kw", [dict(), dict(accumulate=True), dict(wide=False), dict(dtype="f16"),
                                dict(gated=True)])
def test_pairs_that_ask_for_their_next_tile_backward(kw):
    for seed in range(2):
        check_bwd(2100, 2056, 5000 // (2 if kw.get("gated") else 1), seed=seed, **kw)
