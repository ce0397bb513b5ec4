"""What the bindings of the experts' operators refuse, by argument; and two streams that
run them, and the layers' products, at once."""
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from tests.layers_parity import gen, randn

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vocabulary_lm_cross_gb300 import build
    build.build()


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def test_rows():
    ids = torch.zeros((6, 2), dtype=torch.int64, device="cuda")
    order = v.moe_sort(ids, 4)
    x, data = empty(6, 32), empty(order.rows, 32)
    f = torch.float32
    for bad, kind in ((lambda: v.moe_sort(ids.cpu(), 4), TypeError), (lambda: v.moe_sort(ids.float(), 4), TypeError),
                      (lambda: v.moe_sort(ids[0], 4), ValueError), (lambda: v.moe_sort(ids.t(), 4), ValueError),
                      (lambda: v.moe_sort(ids, 0), Exception), (lambda: v.moe_sort(ids, 1025), Exception),
                      (lambda: v.moe_sort(ids, 4, align=0), Exception),
                      (lambda: v.moe_gather(x.to(FP8), order), TypeError), (lambda: v.moe_gather(x[:5], order), ValueError),
                      (lambda: v.moe_gather(x.cpu(), order), TypeError),
                      (lambda: v.moe_gather(x, order, out=data[1:]), ValueError),
                      (lambda: v.moe_gather(x, order, out=data.float()), TypeError),
                      (lambda: v.moe_gather(x, order, fp8=True, out=data), TypeError),
                      (lambda: v.moe_gather(x, order._replace(position=order.position.long())), ValueError),
                      (lambda: v.moe_gather(x, order._replace(offsets=order.offsets[1:])), ValueError),
                      (lambda: v.moe_gather(x, order._replace(counts=order.counts.cpu())), ValueError),
                      (lambda: v.moe_combine(data[1:], order), ValueError),
                      (lambda: v.moe_combine(data, order, empty(6, 3, dtype=f)), ValueError),
                      (lambda: v.moe_combine(data, order, empty(6, 2, dtype=torch.float16)), TypeError),
                      (lambda: v.moe_combine(data, order, empty(2, 6, dtype=f).t()), ValueError),
                      (lambda: v.moe_combine(data, order, None, x.float()), TypeError),
                      (lambda: v.moe_combine(data, order, None, x[:, 1:]), ValueError),
                      (lambda: v.moe_combine(data, order, out=data[:6]), Exception),  # it is read
                      (lambda: v.moe_gather_bwd(data[1:], order), ValueError),
                      (lambda: v.moe_combine_bwd(x, data.float(), order), TypeError),
                      (lambda: v.moe_combine_bwd(x[:, :16], data, order), ValueError),
                      (lambda: v.moe_combine_bwd(x, data, order, want_drows=False, out=data), ValueError),
                      (lambda: v.moe_combine_bwd(x, data, order, want_drows=False, want_dweights=False), Exception),
                      (lambda: v.moe_combine_bwd(x, data, order, out=data), Exception)):
        with pytest.raises(kind):
            bad()


def test_blocks():
    x = empty(64, 256)
    for bad, kind in ((lambda: v.quantize_blocks(x.cpu()), TypeError), (lambda: v.quantize_blocks(x.to(FP8)), TypeError),
                      (lambda: v.quantize_blocks(x[0]), ValueError), (lambda: v.quantize_blocks(x.t()), ValueError),
                      (lambda: v.quantize_blocks(x, rows=False), ValueError),
                      (lambda: v.quantize_blocks(x.expand(3, 64, 256)), Exception)):
        with pytest.raises(kind):
            bad()


def test_products():
    x, w = empty(64, 256, dtype=FP8), empty(128, 256, dtype=FP8)
    f = torch.float32
    xs, ws, off = empty(64, 2, dtype=f), empty(1, 2, dtype=f), torch.zeros(3, dtype=torch.int32, device="cuda")
    w3, ws3 = empty(2, 128, 256, dtype=FP8), empty(2, 1, 2, dtype=f)
    fwd, dw = v.block_linear_fwd, v.block_linear_dweight
    t, ts = empty(96, 256, dtype=FP8), empty(96, 2, dtype=f)
    for bad, kind in ((lambda: fwd(x.bfloat16(), xs, w, ws), TypeError), (lambda: fwd(x, xs, w.half(), ws), TypeError),
                      (lambda: fwd(x, xs, w[:, :128], ws), ValueError), (lambda: fwd(x, xs[:, :1], w, ws), ValueError),
                      (lambda: fwd(x, xs, w, ws[:, :1]), ValueError), (lambda: fwd(x, xs.half(), w, ws), TypeError),
                      (lambda: fwd(x, xs, w, ws, out_dtype=f), TypeError), (lambda: fwd(x, xs, w3, ws3), ValueError),
                      (lambda: fwd(x, xs, w, ws, offsets=off), ValueError),
                      (lambda: fwd(x, xs, w3, ws3, offsets=off.long()), TypeError),
                      (lambda: fwd(x, xs, w3, ws3, offsets=off[:1]), ValueError),
                      (lambda: fwd(x, xs, w3, ws3, offsets=torch.zeros(4, dtype=torch.int32, device="cuda")), ValueError),
                      (lambda: fwd(x, xs, empty(3, 128, 256, dtype=FP8)[::2], ws3, offsets=off), ValueError),
                      (lambda: fwd(x, xs, w, ws, empty(64, 127)), ValueError),
                      (lambda: fwd(x, xs, w, ws, empty(64, 128), out=empty(64, 128, dtype=torch.float16)), TypeError),
                      (lambda: fwd(x, xs, w, ws, out=empty(63, 128)), ValueError),
                      (lambda: fwd(x[:, 1:129], xs[:, :1], w[:, :128], ws[:, :1]), Exception),  # 16-byte aligned rows
                      (lambda: fwd(x, xs, w, ws, dev_err=torch.zeros(1, device="cuda")), TypeError),
                      (lambda: dw(t, ts, x.bfloat16(), xs), TypeError), (lambda: dw(t[:, :128], ts, x, xs), ValueError),
                      (lambda: dw(t, ts, x, xs[:, :1]), ValueError), (lambda: dw(t, ts, x, xs, accumulate=True), ValueError),
                      (lambda: dw(t, ts, x, xs, dweight=empty(96, 63, dtype=f)), ValueError),
                      (lambda: dw(t, ts, x, xs, dweight=empty(96, 64), accumulate=True), Exception),
                      (lambda: dw(t, ts, x, xs, dweight=empty(96, 64, dtype=f), dweight_dtype=torch.bfloat16), TypeError),
                      (lambda: dw(t, ts, x, xs, offsets=off, dweight=empty(96, 64, dtype=f)), ValueError)):
        with pytest.raises(kind):
            bad()
    torch.cuda.synchronize()


def test_two_streams_at_once():
    """Both streams' kernels share the SMs, their tensor memory among them."""
    g = gen(21)
    H, n, E = 512, 640, 8
    up = v.quantize_blocks(randn(g, (n, H), torch.bfloat16, sigma=0.05), square=True)
    ups = v.quantize_blocks((torch.randn((E, n, H), generator=g) * 0.05).bfloat16().cuda(), square=True, transposed=True)
    plain = randn(g, (n, H), torch.bfloat16, sigma=0.05)
    xs = [randn(g, (t, H), torch.bfloat16) for t in (3, 100, 900, 2500)]
    ids = [torch.randint(0, E, (x.shape[0], 2), generator=g).cuda() for x in xs]

    def step(x, ids):
        order = v.moe_sort(ids, E, align=128)
        r = v.moe_gather(x, order, out=torch.zeros((order.rows, H), dtype=x.dtype, device="cuda")).rows
        a = v.quantize_blocks(r, transposed=True)
        z = v.block_linear_fwd(a.q, a.scale, ups.q, ups.scale, offsets=order.offsets,
                               out=torch.zeros((order.rows, n), dtype=x.dtype, device="cuda"))
        d = v.quantize_blocks(z, transposed=True)
        q = v.quantize_blocks(x)
        return (z, v.block_linear_dweight(d.qt, d.scale_t, a.qt, a.scale_t, offsets=order.offsets),
                v.block_linear_fwd(q.q, q.scale, up.q, up.scale), v.linear_fwd(x, plain).y,
                v.moe_combine(z, order))

    want = [step(x, i) for x, i in zip(xs, ids)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for turn in range(12):
        for k, s in enumerate(streams):
            i = (turn + 2 * k) % len(xs)
            with torch.cuda.stream(s):
                got.append((i, step(xs[i], ids[i])))
    torch.cuda.synchronize()
    for i, r in got:
        for a, b in zip(r, want[i]):
            assert torch.equal(a, b)
    v.check_device_errors()
