"""Products of the linear and gated layers on small integers: every product and partial
sum is an integer (or a multiple of a small power of two) that fp32 holds, so
accumulation is exact in any order and the results equal a plain 64-bit evaluation,
rounded once, bit for bit.  A missing, doubled or misplaced element of K, or a tile
handed out wrongly, shows at any size.  describe_linear_plan tells that each way of
running a product is among the cases; one that a change of the estimates moves
elsewhere needs another size here."""
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
    assert torch.equal(want64.float().double(), want64)  # else the case is not exact
    want = want64.to(got.dtype)
    assert torch.equal(got, want), (int((got != want).sum()), (got != want).nonzero()[0].tolist())


def scales(g, n):
    """1/2 or 1: products with them are exact."""
    return torch.exp2(-torch.randint(0, 2, (n,), generator=g, device="cuda").float())


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


def check_glu_fwd(T, K, n, dtype, seed=0):
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


def plan(T, K, N, dtype, want, **kw):
    """The plan, with the fields in `want` checked: rounds (0, 1 or 2 for more), shared
    (whether CTAs share a tile's K), several (pairs take more than one tile) and
    least (tokens a tile)."""
    p = v.describe_linear_plan(T, N, K, DT[dtype], **kw)
    got = dict(kernel=p.kernel, per_sm=p.per_sm, rounds=min(p.exchanges, 2), shared=p.split > 1,
               several=p.tiles > 76, dealt=p.dealt, outputs=p.outputs)
    assert p.tokens >= want.get("least", 0), p
    assert {k: got[k] for k in want if k != "least"} == {k: x for k, x in want.items() if k != "least"}, p


def small(least, per_sm=1, rounds=None):
    """One CTA a tile, or with `rounds` several."""
    d = dict(kernel="small", least=least, per_sm=per_sm, shared=rounds is not None)
    if rounds is not None:
        d["rounds"] = rounds
    return d


def pairs(outputs, dealt, several=True):
    return dict(kernel="pairs", outputs=outputs, dealt=dealt, several=several)


@pytest.mark.parametrize("dtype,T,K,N,want", [
    ("bf16", 1, 264, 127, small(16)), ("bf16", 1, 264, 20480, small(16, 2)),
    ("bf16", 50, 1000, 12300, small(64)), ("f16", 50, 1000, 20480, small(64, 2)),
    ("f16", 300, 1000, 5000, small(112)), ("bf16", 300, 2056, 12300, small(112, 2)),
    ("bf16", 300, 6224, 8200, small(160)), ("bf16", 300, 4112, 20480, small(160, 2)),
    ("bf16", 1, 1000, 127, small(16, 1, 0)), ("bf16", 1, 8208, 5000, small(16, 2, 0)),
    ("f16", 17, 4112, 12300, small(32, 2, 1)), ("bf16", 300, 1000, 127, small(64, 1, 1)),
    ("bf16", 333, 6224, 3918, small(112, 2, 1)), ("bf16", 700, 1000, 127, small(112, 1, 2)),
    ("bf16", 200, 15600, 5000, small(208, 2, 2)), ("f16", 333, 15600, 2056, small(176, 2, 2)),
    ("bf16", 3000, 4112, 300, small(256, 1, 1)), ("bf16", 1500, 15600, 1031, small(256, 2, 2)),
    ("bf16", 300, 264, 20480, pairs(256, True)), ("f16", 300, 2056, 20480, pairs(256, False)),
    ("bf16", 1281, 264, 3077, pairs(128, True)), ("bf16", 1281, 2056, 3077, pairs(128, False)),
    ("e4m3", 50, 1008, 20480, small(64, 2)), ("e4m3", 300, 4112, 5000, small(112)),
    ("e4m3", 300, 4112, 12300, small(112, 2)), ("e4m3", 300, 6224, 20480, small(160, 2)),
    ("e4m3", 1, 6224, 12300, small(16, 2, 0)), ("e4m3", 50, 8208, 12300, small(64, 2, 1)),
    ("e4m3", 300, 15600, 5000, small(160, 2, 1)), ("e4m3", 2100, 15600, 1031, small(224, 2, 2)),
    ("e4m3", 700, 15600, 2056, small(176, 2, 2)), ("e4m3", 300, 272, 20480, pairs(256, True)),
    ("e4m3", 300, 4112, 20480, pairs(256, False)), ("e4m3", 1281, 4112, 3077, pairs(128, False)),
])
def test_every_way_of_running_a_linear_layer(dtype, T, K, N, want):
    plan(T, K, N, dtype, want)
    check_linear_fwd(T, K, N, dtype)
    check_linear_fwd(T, K, N, dtype, seed=1, in_place=True)
    check_linear_fwd(T, K, N, dtype, seed=2, residual=False)


@pytest.mark.parametrize("dtype,T,K,n,want", [
    ("bf16", 1, 264, 8200, small(16)), ("bf16", 1, 264, 20480, small(16, 2)),
    ("bf16", 50, 264, 12300, small(64)), ("bf16", 50, 1000, 20480, small(64, 2)),
    ("bf16", 300, 1000, 5000, small(112)), ("bf16", 300, 2056, 12300, small(112, 2)),
    ("bf16", 2100, 2056, 1031, small(176)), ("bf16", 200, 4112, 12300, small(208)),
    ("bf16", 1, 1000, 3000, small(16, 1, 0)), ("bf16", 1, 1000, 127, small(16, 1, 1)),
    ("bf16", 1, 6224, 12300, small(16, 2, 1)), ("bf16", 90, 6224, 12300, small(96, 2, 2)),
    ("bf16", 700, 2056, 127, small(112, 1, 1)), ("bf16", 300, 8208, 5000, small(112, 2, 2)),
    ("bf16", 3000, 4112, 127, small(208, 1, 2)), ("bf16", 3000, 15600, 300, small(256, 1, 2)),
    ("bf16", 1, 264, 127, pairs(64, True, False)), ("bf16", 1500, 2056, 127, pairs(64, False, False)),
    ("bf16", 33, 264, 20480, pairs(128, True)), ("bf16", 129, 2056, 20480, pairs(128, False)),
    ("e4m3", 1, 272, 12300, small(16)), ("e4m3", 50, 2064, 20480, small(64, 2)),
    ("e4m3", 300, 2064, 5000, small(112)), ("e4m3", 300, 4112, 12300, small(112, 2)),
    ("e4m3", 1, 1008, 2056, small(16, 1, 0)), ("e4m3", 300, 15600, 5000, small(112, 2, 2)),
    ("e4m3", 3000, 8208, 127, small(208, 1, 2)), ("e4m3", 17, 272, 20480, pairs(128, True)),
    ("e4m3", 1500, 4112, 127, pairs(64, False, False)), ("e4m3", 129, 4112, 20480, pairs(128, False)),
])
def test_every_way_of_running_a_gated_layer(dtype, T, K, n, want):
    plan(T, K, n, dtype, want, gated=True)
    check_glu_fwd(T, K, n, dtype)


def grads(kind, dealt, several=True, **kw):
    """kind: the kernel of dx; dealt, several: the pair kernel's tiles."""
    return dict(kernel=kind, dealt=dealt, several=several, **kw)


@pytest.mark.parametrize("gated,T,K,N,want", [
    (False, 1, 264, 20480, grads("small", True, least=16, per_sm=1, rounds=0)),
    (False, 1, 4112, 20480, grads("small", True, least=16, per_sm=2, rounds=0)),
    (False, 50, 1000, 12300, grads("small", True, least=64, rounds=1)),
    (False, 129, 2056, 8200, grads("small", True, least=144, rounds=1)),
    (False, 333, 2056, 20480, grads("small", True, least=176, per_sm=2, rounds=2)),
    (False, 1007, 1000, 12300, grads("small", True, least=256, rounds=1)),
    (False, 2100, 264, 20480, grads("small", False, least=176, per_sm=2, rounds=2)),
    (False, 257, 4112, 1900, grads("pairs", True)),
    (False, 2100, 4112, 300, grads("pairs", False)),
    (True, 300, 1040, 3918, grads("small", True, least=112, rounds=1)),
    (True, 333, 2056, 8200, grads("small", True, least=176, per_sm=2, rounds=2)),
    (True, 3000, 264, 12300, grads("small", False, least=256, per_sm=2, rounds=2)),
    (True, 1500, 4112, 300, grads("pairs", True)),
    (True, 257, 2056, 1900, grads("pairs", False)),
])
def test_every_way_of_running_the_gradients(gated, T, K, N, want):
    plan(T, K, N, "bf16", want, gated=gated, backward=True)
    check_bwd(T, K, N, gated=gated)
    check_bwd(T, K, N, gated=gated, seed=1, accumulate=True)
    check_bwd(T, K, N, gated=gated, seed=2, wide=False)
    check_bwd(T, K, N, gated=gated, seed=3, dtype="f16")


@pytest.mark.parametrize("dtype,finite", [("f16", False), ("bf16", True)])
def test_pre_activation_gradients_have_the_range_of_their_type(dtype, finite):
    x = torch.full((2, 8), 2.0 ** -8, device="cuda").to(DT[dtype])
    w = torch.full((16, 8), 2.0 ** -8, device="cuda").to(DT[dtype])
    z = torch.ones((2, 16), device="cuda").to(DT[dtype])
    z[:, 8:] = 256
    for dy, ok in ((128.0, True), (256.0, finite)):  # dy u = 2^15, and 2^16 > 65504
        d = torch.full((2, 8), dy, device="cuda").to(DT[dtype])
        d[1] = 1
        g = v.glu_bwd(d, x, w, z, act="relu")
        assert torch.isfinite(g.dx[1]).all() and torch.isfinite(g.dweight[8:]).all()
        assert bool(torch.isfinite(g.dx[0]).all()) == ok
        assert bool(torch.isfinite(g.dweight[:8]).all()) == ok
        # below the type's range: zero, without a trace in the sums
        d.fill_(2.0 ** -24)
        small = torch.full_like(z, 0.25)
        assert bool((v.glu_bwd(d, x, w, small, act="relu").dweight == 0).all()) == (dtype == "f16")


def test_plan_refuses():
    for kw in (dict(T=0), dict(N=0), dict(K=60), dict(K=72, dtype=torch.float8_e4m3fn), dict(T=1 << 31),
               dict(dtype=torch.float32), dict(dtype=torch.float8_e4m3fn, backward=True)):
        with pytest.raises(v.capi.VlmceError):
            v.describe_linear_plan(**{**dict(T=4, N=8, K=64, dtype=torch.bfloat16), **kw})
