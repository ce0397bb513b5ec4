"""The products of e4m3 operands with one scale per block of 128, against the fp64 oracle
on the GPU.

Bound before the one rounding: a block's sum of 128 products comes from the tensor core
with fp32 accumulators, in any order and with truncating or rounding additions, (128 + 8)
2^-23 of the terms' magnitudes; the product of the two scales and its product with the sum
2^-24 each; the sum over nb blocks nb 2^-24 more; the residual's addition 2^-24 of all.  So
(140 + nb) 2^-23 of the magnitudes of terms and residual covers it.
"""
import numpy as np
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from oracle import moe as om
from tests.layers_parity import DT, E23, close, f64, gen, randn
from vocabulary_lm_cross_gb300 import capi

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vocabulary_lm_cross_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _no_errors():
    yield
    v.check_device_errors()


def blocks(n):
    return -(-n // 128)


def e4m3(g, rows, cols, pad=0, lead=()):
    """Values of e4m3 in rows whole 16-byte units apart, NaNs behind each row."""
    ld = (cols + 15) // 16 * 16 + 16 * pad
    store = torch.full((*lead, rows, ld), float("nan"))
    store[..., :cols] = torch.randn((*lead, rows, cols), generator=g) * 2
    return store.to(FP8).cuda()[..., :cols]


def scales(g, rows, n, pad=0, lead=()):
    store = torch.full((*lead, rows, n + pad), float("nan"))
    store[..., :n] = torch.exp(torch.randn((*lead, rows, n), generator=g))
    return store.cuda()[..., :n]


def bound(size, K):
    return (140 + blocks(K)) * E23 * size


def near(got, want, dtype, e, what):
    """close(), where the type's range lets it: fp16 ends at 65504, and what is at or above
    65504 + 16 = 65520 (half a step of 2^5 on) rounds to an infinity, nothing below does.
    An element whose exact value is within e of 65520 or above may be that infinity, and one
    at e or more above it has to be."""
    if dtype == "f16":
        e = np.broadcast_to(e, want.shape)
        inf = np.isinf(f64(got)) & (np.abs(want) + e >= 65520) & (np.sign(f64(got)) == np.sign(want))
        assert inf[np.abs(want) - e >= 65520].all(), what
        got = torch.where(torch.from_numpy(inf).to(got.device), torch.zeros_like(got), got)
        want, e = np.where(inf, 0.0, want), np.where(inf, 0.0, e)
    close(got, want, dtype, e, what)


def check_dense(T, N, K, dtype="bf16", by_row=False, residual=False, pad=0, seed=0):
    g = gen(seed + T * 7 + N * 3 + K)
    x, xs = e4m3(g, T, K, pad), scales(g, T, blocks(K), pad)
    w, ws = e4m3(g, N, K, pad), scales(g, N if by_row else blocks(N), blocks(K), pad)
    y, size = om.product(f64(x.float()), f64(xs), f64(w.float()), f64(ws), 1 if by_row else 128)
    res = randn(g, (T, N), DT[dtype], sigma=10.0, pad=pad) if residual else None
    if residual:
        y, size = y + f64(res), size + np.abs(f64(res))
    store = torch.full((T + 1, N + pad), 7.0, dtype=DT[dtype], device="cuda")
    got = v.block_linear_fwd(x, xs, w, ws, res, out=store[:T, :N])
    near(got, y, dtype, bound(size, K), "y")
    assert (store[T:] == 7.0).all() and (store[:, N:] == 7.0).all()
    if residual:
        again = v.block_linear_fwd(x, xs, w, ws, res, out=res)
        assert torch.equal(again, got)
    else:
        assert torch.equal(v.block_linear_fwd(x, xs, w, ws, out_dtype=DT[dtype]), got)


SMALL = [(1, 1, 1), (1, 128, 128), (1, 4096, 2048), (1, 100, 16), (2, 300, 640), (3, 129, 200), (16, 256, 4096),
         (17, 257, 1000), (40, 1000, 136), (64, 136, 16384), (100, 512, 512), (128, 8, 100), (129, 96, 1664),
         (8, 20000, 256),
         # K shared by clusters of two to eight, with each tile
         (1, 12000, 2048), (1, 7500, 1024), (5, 3000, 2048), (20, 7500, 2048), (33, 5000, 2048), (130, 1500, 2048),
         (100, 7500, 2048), (200, 1500, 2048), (200, 500, 2048),
         (40, 5000, 4096), (100, 2000, 2048), (900, 300, 4096), (200, 2000, 4096), (900, 96, 4096), (20, 3000, 4096)]
PAIRS = [(193, 8, 16), (256, 256, 128), (257, 264, 640), (300, 1001, 200), (512, 128, 4096), (700, 777, 1000),
         (1024, 100, 136), (2000, 520, 256),
         (2000, 2600, 264), (513, 9000, 136), (130, 12000, 512),
         (2000, 7777, 16), (1000, 2600, 264), (2600, 1001, 264), (300, 9000, 264), (257, 9000, 400), (4100, 520, 264),
         (3100, 777, 264)]


@pytest.mark.parametrize("by_row", [False, True])
@pytest.mark.parametrize("T,N,K", SMALL + PAIRS)
def test_dense(T, N, K, by_row):
    check_dense(T, N, K, "f16" if (T + N) % 2 else "bf16", by_row, residual=T % 3 == 1, pad=(N + T) % 3)


@pytest.mark.parametrize("T,N,K", [(1, 256, 512), (5, 1000, 4096), (30, 128, 1024), (60, 300, 300), (130, 130, 130),
                                   (300, 1000, 264), (333, 77, 300), (1000, 2600, 264)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_residual_at_any_alignment(T, N, K, dtype):
    for pad in (0, 1, 8):
        check_dense(T, N, K, dtype, residual=True, pad=pad, seed=5)


def test_both_kernels_every_tile_and_split_are_reached():
    plans = [v.describe_block_linear_plan(T, N, K) for T, N, K in SMALL + PAIRS]
    assert {p.kernel for p in plans} == {"pairs", "small"}
    assert {p.rows for p in plans if p.kernel == "small"} == {16, 32, 64, 128}
    assert {1, 2, 4, 8} <= {p.split for p in plans}
    assert {p.per_stage for p in plans if p.kernel == "small"} == {1, 2}


def group_rows(g, E, most, align=1):
    """Rows of each expert: some without any, one with most of them."""
    n = torch.randint(0, most + 1, (E,), generator=g)
    n[torch.rand(E, generator=g) < 0.3] = 0
    n[E // 2] = 3 * most + 1
    return ((n + align - 1) // align * align).tolist()


EXPERTS = [(4, 3, 96, 128), (7, 20, 300, 256), (33, 9, 136, 640), (64, 1, 512, 384), (5, 100, 264, 1000),
           (16, 50, 1000, 200), (3, 700, 264, 512), (2, 1000, 100, 136), (1000, 1, 64, 128), (3, 1400, 1000, 600), (40, 60, 1000, 384),
           (6, 150, 2000, 384), (10, 130, 1200, 256), (6, 60, 2000, 1000), (8, 130, 1000, 1000), (5, 900, 777, 512),
           (4, 900, 2100, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("E,most,N,K", EXPERTS)
def test_experts(E, most, N, K, dtype):
    g = gen(E + N)
    n = group_rows(g, E, most)
    lead = 3 if E % 2 else 0  # rows before the first expert's
    off = np.cumsum([lead] + n)
    T = int(off[-1]) + 5
    by_row, pad = E % 3 == 1, E % 2
    x, xs = e4m3(g, T, K, pad), scales(g, T, blocks(K), pad)
    x[off[-1]:] = float("nan")
    w, ws = e4m3(g, N, K, 0, (E,)), scales(g, N if by_row else blocks(N), blocks(K), 0, (E,))
    offsets = torch.from_numpy(off).int().cuda()
    out = torch.full((T, N), 7.0, dtype=DT[dtype], device="cuda")
    res = randn(g, (T, N), DT[dtype], sigma=5.0) if E % 2 else None
    got = v.block_linear_fwd(x, xs, w, ws, res, offsets=offsets, out=out)
    want, size = np.full((T, N), 7.0), np.zeros((T, N))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want[r], size[r] = om.product(f64(x[r].float()), f64(xs[r]), f64(w[e].float()), f64(ws[e]), 1 if by_row else 128)
    if res is not None:
        used = slice(off[0], off[-1])
        want[used] += f64(res)[used]
        size[used] += np.abs(f64(res)[used])
    near(got, want, dtype, bound(size, K), "y")
    assert (got[off[-1]:] == 7.0).all() and (got[:lead] == 7.0).all()


def test_the_experts_sizes_reach_both_kernels():
    plans = []
    for E, most, N, K in EXPERTS:
        n = group_rows(gen(E + N), E, most)
        plans.append(v.describe_block_linear_plan(sum(n) + 5 + (3 if E % 2 else 0), N, K, E))
    assert {p.kernel for p in plans} == {"pairs", "small"}
    assert {16, 64, 128} <= {p.rows for p in plans}


@pytest.mark.parametrize("E", [1, 8, 1000])
def test_experts_without_any_rows(E):
    g = gen(E)
    x, xs = e4m3(g, 300, 256), scales(g, 300, 2)
    w, ws = e4m3(g, 128, 256, 0, (E,)), scales(g, 1, 2, 0, (E,))
    out = torch.full((300, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v.block_linear_fwd(x, xs, w, ws, offsets=torch.zeros(E + 1, dtype=torch.int32, device="cuda"), out=out)
    assert (out == 7.0).all()
    few = torch.full((2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    v.block_linear_fwd(x[:2], xs[:2], w, ws, offsets=torch.zeros(E + 1, dtype=torch.int32, device="cuda"), out=few)
    assert (few == 7.0).all()


@pytest.mark.parametrize("T", [20, 700])
@pytest.mark.parametrize("bad", [[0, -1, 5, 9], [0, 8, 4, 9], [0, 4, 9, 10 ** 6], [-5, 0, 3, 4]])
def test_offsets_that_are_none_are_reported(T, bad):
    g = gen(3)
    x, xs = e4m3(g, T, 256), scales(g, T, 2)
    w, ws = e4m3(g, 64, 256, 0, (3,)), scales(g, 1, 2, 0, (3,))
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    v.block_linear_fwd(x, xs, w, ws, offsets=off, out=out, dev_err=err)
    assert int(err) == capi.DEVERR_OFFSETS and (out == 7.0).all()
    v.block_linear_fwd(x, xs, w, ws, offsets=off, out=out)
    with pytest.raises(RuntimeError, match="offsets"):
        v.check_device_errors()


# ------------------------------------------------------------ the weight's gradient
def check_dweight(N, K, n, dtype="f32", accumulate=False, pad=0, grouped=True):
    """n: rows of each expert (multiples of 128 but for a last one's that ends with R)."""
    off = np.cumsum([0] + n)
    R = int(off[-1])
    E = len(n)
    g = gen(N + K + R)
    a, sa = e4m3(g, N, R, pad), scales(g, N, blocks(R), pad)
    b, sb = e4m3(g, K, R, pad), scales(g, K, blocks(R), pad)
    want, size = np.zeros((E, N, K)), np.zeros((E, N, K))
    fa, fb = f64(a.float()), f64(b.float())
    ga, gb = f64(sa), f64(sb)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        c = slice(off[e] // 128, blocks(off[e + 1]))
        if n[e]:
            want[e], size[e] = om.product(fa[:, r], ga[:, c], fb[:, r], gb[:, c], 1)
    kw = {"offsets": torch.from_numpy(off).int().cuda()} if grouped else {}
    if not grouped:
        want, size = want[0], size[0]
    start = None
    if accumulate:
        start = torch.randn(want.shape, generator=g).cuda()
        want, size = want + f64(start), size + np.abs(f64(start))
        kw["dweight"] = start.clone()
    got = v.block_linear_dweight(a, sa, b, sb, dweight_dtype=DT[dtype], accumulate=accumulate, **kw)
    near(got, want, dtype, bound(size, R), "dweight")
    if accumulate:
        for e in range(E):
            if grouped and n[e] == 0:
                assert torch.equal(got[e], start[e])


SIZES = [(8, 16, [128]), (256, 256, [256, 0, 128]), (300, 264, [0, 384, 128, 0]), (129, 1001, [128, 128]),
         (1000, 130, [0, 0, 640]), (64, 40, [128] * 40), (520, 776, [1280, 0, 0, 256, 128])]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N,K,n", SIZES)
def test_dweight_of_experts(N, K, n, accumulate):
    check_dweight(N, K, n, accumulate=accumulate, pad=N % 2)


@pytest.mark.parametrize("K", [288, 352, 416])
def test_dweight_of_experts_without_rows_after_others(K):
    """A warp's last store of a tile still reads its buffer when a tile without any products
    follows at once, also where a tile has an odd number of stores."""
    for N in (256, 200):
        check_dweight(N, K, [128] * 38 + [0] * 38 + [128] * 38 + [0] * 38)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,n", SIZES)
def test_dweight_in_16_bits(N, K, n, dtype):
    check_dweight(N, K, n, dtype)


@pytest.mark.parametrize("R", [1, 16, 100, 128, 257, 1000, 4000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_dweight_dense_and_with_a_ragged_end(R, accumulate):
    check_dweight(200, 136, [R], accumulate=accumulate, grouped=False)
    if R > 128:
        check_dweight(40, 264, [128, R - 128], accumulate=accumulate)


def test_dweight_of_no_rows_and_of_bad_offsets():
    a, sa = torch.empty((64, 0), dtype=FP8, device="cuda"), torch.empty((64, 0), device="cuda")
    assert (v.block_linear_dweight(a, sa, a, sa) == 0).all()
    keep = torch.ones((64, 64), device="cuda")
    v.block_linear_dweight(a, sa, a, sa, dweight=keep, accumulate=True)
    assert (keep == 1).all()
    g = gen(1)
    b, sb = e4m3(g, 64, 512), scales(g, 64, 4)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in ([0, 100, 512], [128, 64, 512], [0, 256, 640], [16, 128, 256]):
        err.zero_()
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        r = v.block_linear_dweight(b, sb, b, sb, offsets=off, dev_err=err)
        assert int(err) == capi.DEVERR_OFFSETS and (r == 0).all()
        keep = torch.ones((2, 64, 64), device="cuda")
        v.block_linear_dweight(b, sb, b, sb, offsets=off, dev_err=err, dweight=keep, accumulate=True)
        assert (keep == 1).all()


def test_nan_and_zero_scales_stay_in_their_rows():
    g = gen(2)
    for T in (20, 400):
        x, xs = e4m3(g, T, 512), scales(g, T, 4)
        w, ws = e4m3(g, 300, 512), scales(g, 3, 4)
        want = v.block_linear_fwd(x, xs, w, ws)
        xs = xs.contiguous()
        xs[3, 2], xs[7] = float("nan"), 0.0
        got = v.block_linear_fwd(x, xs, w, ws)
        assert torch.isnan(got[3]).all() and (got[7] == 0).all()
        keep = [i for i in range(T) if i not in (3, 7)]
        assert torch.equal(got[keep], want[keep])


def test_streams_and_graphs():
    g = gen(4)
    T, N, K, E = 400, 264, 512, 6
    x, xs = e4m3(g, T, K), scales(g, T, 4)
    w, ws = e4m3(g, N, K, 0, (E,)), scales(g, 3, 4, 0, (E,))
    d, sd = e4m3(g, N, 512), scales(g, N, 4)
    e, se = e4m3(g, 136, 512), scales(g, 136, 4)
    off = torch.tensor([0, 30, 30, 100, 101, 350, 400], dtype=torch.int32, device="cuda")
    cut = torch.tensor([0, 128, 128, 512], dtype=torch.int32, device="cuda")

    def step():
        return (v.block_linear_fwd(x, xs, w, ws, offsets=off), v.block_linear_fwd(x, xs, w[0], ws[0]),
                v.block_linear_fwd(x[:9], xs[:9], w[1], ws[1]), v.block_linear_dweight(d, sd, e, se, offsets=cut))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    off.copy_(torch.tensor([0, 0, 5, 205, 390, 400, 400], dtype=torch.int32))
    cut.copy_(torch.tensor([0, 256, 384, 512], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_outputs_and_rows_beyond_2_to_the_31_elements():
    g = gen(6)
    N, K = 16384, 256
    T = 2 ** 31 // N + 300
    x, xs = e4m3(g, 300, K), scales(g, 300, 2)
    w, ws = e4m3(g, N, K), scales(g, N // 128, 2)
    far = torch.zeros((T, K), dtype=FP8, device="cuda")
    fars = torch.ones((T, 2), device="cuda")
    far[-300:], fars[-300:] = x, xs
    want = v.block_linear_fwd(x, xs, w, ws)
    got = v.block_linear_fwd(far, fars, w, ws)
    # (another kernel sums the same two blocks in the same order)
    assert torch.equal(got[-300:], want) and not got[:128].any()
    off = torch.tensor([0, 5, T - 300, T], dtype=torch.int32, device="cuda")
    y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    v.block_linear_fwd(far, fars, w.expand(3, N, K).contiguous(), ws.expand(3, N // 128, 2).contiguous(), offsets=off,
                       out=y)
    assert torch.equal(y[-300:], want)


def test_a_gradient_beyond_2_to_the_31_elements():
    g = gen(7)
    N, K, E = 8192, 8192, 34
    d, sd = e4m3(g, N, 256), scales(g, N, 2)
    e, se = e4m3(g, K, 256), scales(g, K, 2)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E - 1:] = torch.tensor([128, 256], dtype=torch.int32)
    got = v.block_linear_dweight(d, sd, e, se, offsets=off, dweight_dtype=torch.bfloat16)
    last = v.block_linear_dweight(d[:, 128:], sd[:, 1:], e[:, 128:], se[:, 1:], dweight_dtype=torch.bfloat16)
    assert torch.equal(got[-1], last) and not got[:E - 2].any() and got[E - 2].any()
