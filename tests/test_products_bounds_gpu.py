"""The linear and gated layers write their outputs' elements and nothing beside them: rows
of any length in buffers whose strides and bases the widest stores accept, the memory
between and after the rows as it was.  Exact values as in test_products_exact_gpu.py."""
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from tests.test_products_exact_gpu import DT, gen, ints, same, scales

pytestmark = pytest.mark.gpu


class Framed:
    """[rows, cols] in a buffer of a known pattern; ld and offset in elements."""

    def __init__(self, rows, cols, ld, offset=8, dtype=torch.bfloat16, init=None):
        n = offset + rows * ld + 64
        self.store = (torch.arange(n, device="cuda") % 251 + 1).to(torch.int16).view(dtype)
        self.before = self.store.clone()
        self.t = self.store.as_strided((rows, cols), (ld, 1), offset)
        self.around = torch.ones(n, dtype=torch.bool, device="cuda")
        self.around.as_strided((rows, cols), (ld, 1), offset).fill_(False)
        if init is not None:
            self.t.copy_(init)

    def check(self):
        now, was = self.store.view(torch.int16)[self.around], self.before.view(torch.int16)[self.around]
        assert torch.equal(now, was), int((now != was).sum())


def up8(n):
    return (n + 7) // 8 * 8


# rows that end in every place of a 16-byte unit, of one to several tiles
ENDS = [1, 5, 7, 8, 9, 12, 15, 31, 60, 62, 65, 67, 124, 127, 129, 188, 250, 255, 257, 1030, 1031, 1037]


@pytest.mark.parametrize("T,K", [(300, 32), (2100, 144), (2100, 1008), (1, 1008), (70, 1008)])
@pytest.mark.parametrize("N", ENDS)
def test_linear_layer(N, T, K):
    for dtype, extra in (("bf16", 0), ("f16", 40), ("e4m3", 8)):
        g = gen(N)
        x, w = ints(g, (T, K), dtype=dtype), ints(g, (N, K), dtype=dtype)
        odt = "bf16" if dtype == "e4m3" else dtype
        z = x.double() @ w.double().t()
        kw = {}
        if dtype == "e4m3":
            kw = dict(x_scale=scales(g, T), weight_scale=scales(g, N))
            z = z * kw["x_scale"].double()[:, None] * kw["weight_scale"].double()
        r = ints(g, (T, N), 100, odt)
        y = Framed(T, N, up8(N) + extra, dtype=DT[odt])
        p = Framed(T, N, up8(N) + extra, dtype=DT[odt])
        v.linear_fwd(x, w, None, r, act="relu", preact=p.t, out=y.t, **kw)
        same(p.t, z)
        same(y.t, z.clamp(min=0) + r.double())
        y.check()
        p.check()
        y = Framed(T, N, up8(N) + extra, dtype=DT[odt], init=r)  # residual in place
        v.linear_fwd(x, w, None, y.t, out=y.t, **kw)
        same(y.t, z + r.double())
        y.check()


@pytest.mark.parametrize("T,K", [(300, 32), (2100, 144), (4400, 2064), (1, 1008), (70, 1008)])
@pytest.mark.parametrize("n", ENDS)
def test_gated_layer(n, T, K):
    for dtype, extra in (("bf16", 0), ("e4m3", 8)):
        g = gen(n)
        x, w = ints(g, (T, K), 1, dtype), ints(g, (2 * n, K), 1, dtype)
        z = x.double() @ w.double().t()
        kw = {}
        if dtype == "e4m3":
            kw = dict(x_scale=scales(g, T), weight_scale=scales(g, 2 * n))
            z = z * kw["x_scale"].double()[:, None] * kw["weight_scale"].double()
        y = Framed(T, n, up8(n) + extra)
        # gate and up side by side: where 2n is whole units and n is not, the gate's last
        # unit holds the first of up
        for ld in (2 * n, up8(2 * n) + extra):
            p = Framed(T, 2 * n, ld)
            for _ in range(3):
                v.glu_fwd(x, w, act="relu", preact=p.t, out=y.t, **kw)
                same(p.t, z)
                same(y.t, z[:, :n].clamp(min=0) * z[:, n:])
            y.check()
            p.check()


@pytest.mark.parametrize("T,K,N", [(300, 40, 77), (700, 264, 1031), (2100, 2056, 300), (1, 264, 2050)])
def test_gradients(T, K, N):
    g = gen(N)
    x, w, dy = ints(g, (T, K)), ints(g, (N, K)), ints(g, (T, N))
    for ld in (K, K + 8):
        dx = Framed(T, K, ld)
        flat = (torch.arange(N * K + 64, device="cuda") % 251 + 1).to(torch.int32).view(torch.float32)
        kept = flat[N * K:].clone()
        v.linear_bwd(dy, x, w, out=dx.t, dweight=flat[:N * K].view(N, K))
        same(dx.t, dy.double() @ w.double())
        same(flat[:N * K].view(N, K), dy.double().t() @ x.double())
        dx.check()
        assert torch.equal(flat[N * K:].view(torch.int32), kept.view(torch.int32))
