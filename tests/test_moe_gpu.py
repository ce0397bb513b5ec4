"""The experts' row operators against the fp64 oracle on the GPU.

Bounds: gather moves values (equal); combine adds k weighted terms and the residual in
fp32, a multiply-add or an addition each, so its error before the one rounding is at most
(k + 2) 2^-24 of the terms' magnitudes; a gradient row is one product rounded to fp32 and
then to the type; dweights sums H products in any order: (H + 8) 2^-24 of their
magnitudes.
"""
import numpy as np
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from oracle import moe as om
from tests.layers_parity import DT, close, f64, gen, randn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vocabulary_lm_cross_gb300 import build
    build.build()


def routing(seed, T, k, E, dropped=False, skew=False, dtype=torch.int64):
    g = gen(seed)
    score = torch.rand((T, E), generator=g)
    if skew:
        score[:, 0] += 1.0  # every token's first choice
        score[:, E // 2:] -= 1.0  # hardly anybody's
    ids = torch.topk(score, min(k, E), dim=1).indices
    if k > E:
        ids = ids.repeat(1, -(-k // E))[:, :k]  # an expert named twice
    if dropped:
        ids[torch.rand((T, k), generator=g) < 0.3] = -1
        ids[torch.rand((T, k), generator=g) < 0.1] = E
    return ids.to(dtype)


def check_order(ids, E, align):
    order = v.moe_sort(ids.cuda(), E, align=align)
    pos, off, cnt = om.sort(ids.numpy(), E, align)
    assert np.array_equal(order.position.cpu().numpy(), pos)
    assert np.array_equal(order.offsets.cpu().numpy(), off)
    assert np.array_equal(order.counts.cpu().numpy(), cnt)
    T, k = ids.shape
    assert off[-1] <= order.rows == (T * k + min(E, T * k) * (align - 1)) // align * align
    return order, pos


@pytest.mark.parametrize("T,k,E,align", [
    (1, 1, 1, 1), (1, 8, 8, 1), (3, 2, 1024, 128), (7, 3, 5, 16), (33, 4, 33, 1), (64, 8, 128, 1),
    (257, 1, 31, 3), (1000, 2, 64, 128), (2049, 1, 7, 1), (5000, 3, 1000, 128), (16384, 8, 256, 128),
    (70000, 2, 17, 1), (5, 64, 64, 1), (9, 6, 2, 1)])
@pytest.mark.parametrize("kind", ["plain", "dropped", "skewed"])
def test_sort(T, k, E, align, kind):
    if T * k > 20000 and kind == "skewed":
        kind = "plain"  # (the oracle is slow)
    ids = routing(T * 31 + E, T, k, E, kind == "dropped", kind == "skewed",
                  torch.int32 if T % 2 else torch.int64)
    check_order(ids, E, align)


def test_sort_of_nothing_of_nobodys_and_of_strided_ids():
    order = v.moe_sort(torch.empty((0, 4), dtype=torch.int64, device="cuda"), 6, align=16)
    assert order.rows == 0 and order.offsets.tolist() == [0] * 7 and order.counts.tolist() == [0] * 6
    check_order(torch.full((100, 2), -1, dtype=torch.int32), 9, 128)
    check_order(torch.full((100, 2), 2 ** 40 + 1, dtype=torch.int64), 9, 1)
    wide = routing(5, 300, 8, 20)
    some = wide.cuda()[:, 2:5]
    pos, off, _ = om.sort(wide[:, 2:5].numpy(), 20, 1)
    order = v.moe_sort(some, 20)
    assert np.array_equal(order.position.cpu().numpy(), pos)
    every = v.moe_sort(wide.cuda()[::3], 20)
    assert np.array_equal(every.position.cpu().numpy(), om.sort(wide[::3].numpy(), 20, 1)[0])


SHAPES = [(1, 1, 1, 1, 1), (1, 8, 8, 4096, 1), (5, 3, 4, 100, 16), (37, 2, 6, 1001, 128), (64, 8, 16, 264, 1),
          (130, 12, 12, 2056, 16), (300, 4, 64, 640, 128),
          (9, 3, 5, 4112, 16), (70, 2, 3, 48, 1), (33, 2, 4, 8200, 1), (20, 8, 16, 100, 1), (20, 6, 16, 1001, 16),
          (11, 5, 9, 30, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,E,H,align", SHAPES)
def test_gather_and_its_gradient(T, k, E, H, align, dtype):
    ids = routing(T + H, T, k, E, dropped=T % 2 == 0)
    order, pos = check_order(ids, E, align)
    g = gen(H)
    x = randn(g, (T, H), DT[dtype], pad=H % 5)
    out = torch.full((order.rows + 2, H), 7.0, dtype=DT[dtype], device="cuda")
    r = v.moe_gather(x, order, out=out[:order.rows])
    want = np.full((order.rows + 2, H), 7.0)
    off, cnt = order.offsets.tolist(), order.counts.tolist()
    for e in range(E):
        want[off[e] + cnt[e]:off[e + 1]] = 0.0  # between two experts' rows; behind the last's as it was
    for t, _, row in om.pairs(pos):
        want[row] = f64(x)[t]
    assert np.array_equal(f64(out), want)
    assert r.rows.data_ptr() == out.data_ptr() and r.scale is None
    drows = randn(g, (order.rows, H), DT[dtype], pad=H % 3)
    dx = v.moe_gather_bwd(drows, order)
    y, size = om.combine(f64(drows), pos)
    close(dx, y, dtype, (k + 2) * U * size, "dx")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,E,H,align", SHAPES)
def test_gather_quantised(T, k, E, H, align, dtype):
    ids = routing(T + H + 1, T, k, E, dropped=T % 2 == 1)
    order, pos = check_order(ids, E, align)
    x = randn(gen(H + 1), (T, H), DT[dtype], sigma=3.0, pad=8 * (H % 2))
    r = v.moe_gather(x, order, fp8=True)
    q = v.quantize_blocks(x)
    assert r.rows.shape == (order.rows, H) and r.scale.shape == (order.rows, -(-H // 128))
    got, scale = r.rows.view(torch.uint8).cpu(), r.scale.cpu()
    want, ws = q.q.view(torch.uint8).cpu(), q.scale.cpu()
    for t, _, row in om.pairs(pos):
        assert torch.equal(got[row], want[t]) and torch.equal(scale[row], ws[t])
    off, cnt = order.offsets.tolist(), order.counts.tolist()
    for e in range(E):
        assert not got[off[e] + cnt[e]:off[e + 1]].any()
        assert torch.isfinite(scale[off[e] + cnt[e]:off[e + 1]]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,E,H,align", SHAPES)
@pytest.mark.parametrize("wide", [True, False])
def test_combine_and_its_gradients(T, k, E, H, align, dtype, wide):
    ids = routing(T + 2 * H, T, k, E, dropped=T % 2 == 0)
    order, pos = check_order(ids, E, align)
    g = gen(H + 2)
    data = randn(g, (order.rows, H), DT[dtype], pad=H % 7)
    if order.rows:  # what no pair has is not read
        free = np.setdiff1d(np.arange(order.rows), pos[pos >= 0])
        data[torch.from_numpy(free).cuda()] = float("nan")
    w = torch.rand((T, k + 3), generator=g).to(torch.float32 if wide else DT[dtype]).cuda()[:, 1:1 + k]
    res = randn(g, (T, H), DT[dtype], sigma=3.0) if wide else None
    y, size = om.combine(np.nan_to_num(f64(data)), pos, f64(w), f64(res) if wide else None)
    close(v.moe_combine(data, order, w, res), y, dtype, (k + 2) * U * size, "y")
    dy = randn(g, (T, H), DT[dtype], pad=H % 2)
    out = torch.full((order.rows + 1, H), 7.0, dtype=DT[dtype], device="cuda")
    r = v.moe_combine_bwd(dy, data, order, w, out=out[:order.rows])
    drows, dw, dsize = om.combine_bwd(f64(dy), np.nan_to_num(f64(data)), pos, f64(w))
    off, cnt = order.offsets.tolist(), order.counts.tolist()
    for e in range(E):
        drows[off[e] + cnt[e]:off[e + 1]] = 0.0
    drows[off[E]:] = 7.0
    close(r.drows, drows, dtype, U * np.abs(drows), "drows")
    assert (out[order.rows:] == 7.0).all()
    close(r.dweights, dw, "f32", (H + 8) * U * dsize, "dweights")
    only = v.moe_combine_bwd(dy, data, order, w, want_drows=False)
    assert only.drows is None and torch.equal(only.dweights, r.dweights)
    rows = v.moe_combine_bwd(dy, data, order, w, want_dweights=False)
    assert rows.dweights is None
    used = torch.from_numpy(np.unique(pos[pos >= 0])).cuda()
    assert torch.equal(rows.drows[used], r.drows[used])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", [16, 30, 100, 264, 1001])
def test_rows_at_any_alignment(H, dtype):
    """x at the end and the start of its memory, 8-bit rows anywhere: as from and to aligned
    rows."""
    T, k, E = 23, 3, 5
    order = v.moe_sort(routing(H, T, k, E).cuda(), E, align=4)
    R = int(order.offsets[-1])
    flat = randn(gen(H), (T * H + 3,), DT[dtype])
    aligned = flat[3:].view(T, H).clone()
    want8, want = v.moe_gather(aligned, order, fp8=True), v.moe_gather(aligned, order).rows
    for x in (flat[3:].view(T, H), torch.cat([flat[3:], flat[:1]])[:-1].view(T, H)):
        got = v.moe_gather(x, order, fp8=True)
        assert torch.equal(got.rows[:R].view(torch.uint8), want8.rows[:R].view(torch.uint8))
        assert torch.equal(got.scale[:R], want8.scale[:R])
        assert torch.equal(v.moe_gather(x, order).rows[:R], want[:R])
        for pad, skip in ((1, 0), (5, 0), (16, 3)):
            store = torch.full((order.rows, H + pad), 77, dtype=torch.uint8, device="cuda")
            out = store[:, skip:skip + H].view(torch.float8_e4m3fn)
            got = v.moe_gather(x, order, fp8=True, out=out)
            assert torch.equal(out[:R].view(torch.uint8), want8.rows[:R].view(torch.uint8))
            assert torch.equal(got.scale[:R], want8.scale[:R])
            assert (store[:, :skip] == 77).all() and (store[:, skip + H:] == 77).all() and (store[R:] == 77).all()


def test_combine_in_place_of_the_residual_and_without_weights():
    order, pos = check_order(routing(3, 50, 4, 9), 9, 1)
    g = gen(9)
    data, res = randn(g, (order.rows, 96), torch.bfloat16), randn(g, (50, 96), torch.bfloat16)
    want = v.moe_combine(data, order, None, res)
    y, size = om.combine(f64(data), pos, None, f64(res))
    close(want, y, "bf16", 6 * U * size, "y")
    got = v.moe_combine(data, order, None, res, out=res)
    assert got.data_ptr() == res.data_ptr() and torch.equal(got, want)


def test_positions_outside_the_rows_are_nobodys():
    order, pos = check_order(routing(4, 20, 2, 5), 5, 1)
    p = order.position.clone()
    p[3, 1], p[7, 0] = order.rows, 2 ** 31 - 1
    bad = order._replace(position=p)
    pos = pos.copy()
    pos[3, 1] = pos[7, 0] = -1
    g = gen(10)
    data = randn(g, (order.rows, 72), torch.float32)
    y, size = om.combine(f64(data), pos)
    close(v.moe_gather_bwd(data, bad), y, "f32", 4 * U * size, "dx")
    x = randn(g, (20, 72), torch.float32)
    out = torch.full((order.rows, 72), 7.0, device="cuda")
    v.moe_gather(x, bad, out=out)
    want = np.full(out.shape, 7.0)
    for t, _, row in om.pairs(pos):
        want[row] = f64(x)[t]
    assert np.array_equal(f64(out), want)


def test_no_tokens():
    order = v.moe_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3)
    x = torch.empty((0, 64), device="cuda")
    assert v.moe_gather(x, order).rows.shape == (0, 64)
    assert v.moe_gather(x, order, fp8=True).scale.shape == (0, 1)
    assert v.moe_combine(x, order).shape == (0, 64)
    r = v.moe_combine_bwd(x, x, order)
    assert r.drows.shape == (0, 64) and r.dweights.shape == (0, 2)


def test_rows_between_are_cleared_without_any_tokens():
    """An order of no tokens whose experts still hold rows: those become zero."""
    empty = v.moe_sort(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 2)
    order = empty._replace(offsets=torch.tensor([0, 3, 4], dtype=torch.int32, device="cuda"), rows=5)
    x = torch.empty((0, 40), device="cuda")
    data = randn(gen(3), (5, 40), torch.float32)
    for call in (lambda out: v.moe_gather(x, order, out=out),
                 lambda out: v.moe_combine_bwd(x, data, order, out=out)):
        out = torch.full((5, 40), 7.0, device="cuda")
        call(out)
        assert torch.equal(out[:4], torch.zeros_like(out[:4])) and bool((out[4] == 7.0).all())


def test_rows_beyond_2_to_the_31_elements():
    H, T = 8192, 4
    R = 2 ** 31 // H + 40
    data = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    position = torch.tensor([[R - 1, 5], [R - 7, R - 2], [0, R - 3], [1, 2]], dtype=torch.int32, device="cuda")
    order = v.MoEOrder(position, torch.tensor([0, R], dtype=torch.int32, device="cuda"),
                       torch.tensor([R], dtype=torch.int32, device="cuda"), R)
    x = randn(gen(1), (T, H), torch.bfloat16)
    v.moe_gather(x, order, out=data)
    assert torch.equal(data[position.long()], x[:, None, :].expand(T, 2, H))
    assert torch.equal(v.moe_gather_bwd(data, order), x * 2)
    r = v.moe_combine_bwd(x, data, order, out=torch.zeros_like(data))
    assert torch.equal(r.drows[position.long()], x[:, None, :].expand(T, 2, H))


def test_streams_and_graphs():
    ids = routing(8, 200, 4, 16).cuda()
    x = randn(gen(11), (200, 512), torch.bfloat16)
    w = torch.rand((200, 4), generator=gen(12)).cuda()

    def step():
        order = v.moe_sort(ids, 16, align=16)
        r = v.moe_gather(x, order)
        y = v.moe_combine(r.rows, order, w, x)
        b = v.moe_combine_bwd(y, r.rows, order, w, out=torch.zeros_like(r.rows))
        return order.position, y, b.drows, b.dweights, v.moe_gather_bwd(b.drows, order)

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
    for other in (routing(9, 200, 4, 16), routing(10, 200, 4, 16, skew=True)):
        ids.copy_(other.cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
