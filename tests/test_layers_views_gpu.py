"""Inputs and outputs that are columns of one buffer, side by side at the same stride: they
share a span of memory and no element."""
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from vocabulary_lm_cross_gb300 import build, capi

gpu = pytest.mark.gpu
P = 1 << 20
BF16 = capi.BF16


def fwd(lib, y, T=4, ys=128, x=P, xs=128, H=64):
    return lib.rmsnorm_fwd(x, xs, None, H, 8 * P, BF16, BF16, T, H, 1e-6, 0.0, y, ys, BF16, None,
                           H, None, None, None)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


# x: rows of 128 bytes, 256 bytes apart
@pytest.mark.parametrize("y,kw", [(P + 2, {}), (P + 126, {}), (P + 254, {}), (P + 256 + 130, {}),
                                  (P - 256 * 3 + 126, {}), (P + 128, dict(ys=64)),
                                  (P + 128, dict(ys=136)), (P + 256, dict(T=2, xs=127)),
                                  (P + 126, dict(T=1))])
def test_shared_elements_are_refused(lib, y, kw):
    assert fwd(lib, y, **kw) == capi.ERR_INVALID_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up")
@pytest.mark.parametrize("y,kw", [(P + 128, {}), (P - 128, {}), (P + 3 * 256 + 128, {}),
                                  (P + 128, dict(T=1)), (P + 4 * 256, {})])
def test_columns_side_by_side_pass_the_checks(lib, y, kw):
    assert fwd(lib, y, **kw) in (capi.ERR_CUDA, capi.ERR_UNSUPPORTED_DEVICE)


def columns(T, widths, dtype=torch.bfloat16, seed=0):
    """Column views of one buffer, random, and the buffer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    store = torch.randn((T, sum(widths)), generator=g, device="cuda").to(dtype)
    return store, store.split(widths, dim=1)


def weight(*shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    return (torch.randn(shape, generator=g, device="cuda") * shape[-1] ** -0.5).bfloat16()


@gpu
@pytest.mark.parametrize("T,H", [(1, 64), (7, 520), (2000, 520), (7, 501), (2000, 2001), (3000, 1001)])
def test_norm(T, H):
    store, (x, r, y, s, dy, dx) = columns(T, [H] * 6)
    w = weight(H)
    keep = store.clone()
    want = v.rmsnorm_fwd(x.contiguous(), w, r.contiguous())
    got = v.rmsnorm_fwd(x, w, r, out=y, residual_out=s)
    tol = dict(rtol=2 ** -7, atol=2 ** -20)  # rows at another alignment take another kernel
    torch.testing.assert_close(y, want.y, **tol)
    assert torch.equal(s, want.residual)
    assert torch.equal(store[:, :2 * H], keep[:, :2 * H]) and torch.equal(store[:, 4 * H:], keep[:, 4 * H:])
    ref = v.rmsnorm_bwd(dy.contiguous(), s.contiguous(), w, got.rstd)
    v.rmsnorm_bwd(dy, s, w, got.rstd, out=dx)
    torch.testing.assert_close(dx, ref.dx, rtol=2 ** -7, atol=2 ** -8 * float(ref.dx.abs().max()))
    assert torch.equal(dy, keep[:, 4 * H:5 * H])


@gpu
@pytest.mark.parametrize("T", [1, 40, 700, 2100])
@pytest.mark.parametrize("N,pad", [(264, 0), (1040, 0), (1031, 9)])
def test_linear(T, N, pad):
    K = 264
    # x and dx start on 16 bytes, as do the rows
    widths = [K, N, N, N, pad + -(K + pad + 3 * N) % 8, K, N, -N % 8]
    store, (x, r, y, z, gap, dx, dy, _) = columns(T, widths)
    w, b = weight(N, K), weight(N)
    keep = store.clone()
    want = v.linear_fwd(x.contiguous(), w, b, r.contiguous(), act="silu", preact=True)
    v.linear_fwd(x, w, b, r, act="silu", preact=z, out=y)
    assert torch.equal(y, want.y) and torch.equal(z, want.preact)
    a, c = K + N, K + 3 * N
    assert torch.equal(store[:, :a], keep[:, :a]) and torch.equal(store[:, c:], keep[:, c:])
    ref = v.linear_bwd(dy.contiguous(), x.contiguous(), w, z.contiguous(), act="silu")
    got = v.linear_bwd(dy, x, w, z, act="silu", out=dx)
    assert torch.equal(got.dweight, ref.dweight) and torch.equal(dx, ref.dx)
    assert torch.equal(dy, keep[:, c + gap.shape[1] + K:][:, :N])
