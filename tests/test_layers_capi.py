"""The decoder-layer entry points refuse bad arguments on the host before anything
is enqueued, and size their workspaces.  CPU only: no compute call is made (fake,
suitably aligned device addresses; every call below fails its checks)."""
import math

import pytest

from vocabulary_lm_cross_gb300 import build, capi

P = 1 << 20
FAR = 1 << 30  # apart from P by more than any buffer here


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


def args(defaults, kw):
    assert set(kw) <= set(defaults), kw
    return [{**defaults, **kw}[k] for k in defaults]


RMS_FWD = dict(x=P, xs=64, res=None, rs=64, w=P, wd=capi.BF16, dt=capi.BF16, T=4, H=64, eps=1e-6,
               off=0.0, y=2 * FAR, ys=64, yd=capi.BF16, ro=None, ros=64, rstd=P, scale=None,
               stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=capi.E4M3, wd=capi.E4M3, yd=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(wd=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(yd=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(T=-1), capi.ERR_INVALID_ARG),
    (dict(H=0), capi.ERR_INVALID_ARG),
    (dict(eps=-1.0), capi.ERR_INVALID_ARG),
    (dict(eps=math.nan), capi.ERR_INVALID_ARG),
    (dict(off=math.inf), capi.ERR_INVALID_ARG),
    (dict(w=None), capi.ERR_INVALID_ARG),
    (dict(x=None), capi.ERR_INVALID_ARG),
    (dict(y=None), capi.ERR_INVALID_ARG),
    (dict(xs=63), capi.ERR_INVALID_ARG),
    (dict(ys=10), capi.ERR_INVALID_ARG),
    (dict(res=FAR, rs=63), capi.ERR_INVALID_ARG),
    (dict(ro=FAR, ros=63), capi.ERR_INVALID_ARG),
    (dict(yd=capi.E4M3), capi.ERR_INVALID_ARG),          # no scale
    (dict(scale=P), capi.ERR_INVALID_ARG),               # scale without e4m3
    (dict(y=P), capi.ERR_INVALID_ARG),                   # y overlaps x
    (dict(y=P + 6 * 64), capi.ERR_INVALID_ARG),           # and in its last row
    (dict(res=2 * FAR), capi.ERR_INVALID_ARG),           # y overlaps the residual
    (dict(ro=2 * FAR), capi.ERR_INVALID_ARG),            # y overlaps residual_out
    (dict(ro=P, ros=72), capi.ERR_INVALID_ARG),          # in place with another stride
    (dict(x=P + 1), capi.ERR_MISALIGNED),
    (dict(y=2 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(w=P + 1), capi.ERR_MISALIGNED),
    (dict(rstd=P + 2), capi.ERR_MISALIGNED),
    (dict(H=(1 << 30) + 1, xs=1 << 31, ys=1 << 31), capi.ERR_TOO_LARGE),
    (dict(T=1 << 31), capi.ERR_TOO_LARGE),
    (dict(xs=1 << 62), capi.ERR_TOO_LARGE),
])
def test_rmsnorm_fwd_refuses(lib, kw, code):
    assert lib.rmsnorm_fwd(*args(RMS_FWD, kw)) == code


RMS_BWD = dict(dy=P, dys=64, x=FAR, xs=64, w=P, wd=capi.BF16, rstd=P, dres=None, drs=64,
               dt=capi.BF16, T=4, H=64, off=0.0, dx=2 * FAR, dxs=64, dw=P, acc=0, ws=P,
               wsb=1 << 20, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(wd=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(T=-1), capi.ERR_INVALID_ARG),
    (dict(rstd=None), capi.ERR_INVALID_ARG),
    (dict(dy=None), capi.ERR_INVALID_ARG),
    (dict(dx=None), capi.ERR_INVALID_ARG),
    (dict(dxs=63), capi.ERR_INVALID_ARG),
    (dict(drs=63, dres=P), capi.ERR_INVALID_ARG),
    (dict(dx=FAR), capi.ERR_INVALID_ARG),                # dx over x
    (dict(dx=P, dxs=72), capi.ERR_INVALID_ARG),          # over dy with another stride
    (dict(off=math.nan), capi.ERR_INVALID_ARG),
    (dict(ws=None), capi.ERR_WORKSPACE_TOO_SMALL),
    (dict(wsb=256), capi.ERR_WORKSPACE_TOO_SMALL),
    (dict(ws=P + 16), capi.ERR_MISALIGNED),
    (dict(dw=P + 2), capi.ERR_MISALIGNED),
    (dict(dx=2 * FAR + 1), capi.ERR_MISALIGNED),
])
def test_rmsnorm_bwd_refuses(lib, kw, code):
    assert lib.rmsnorm_bwd(*args(RMS_BWD, kw)) == code


LINEAR_FWD = dict(x=P, xs=64, xsc=None, w=FAR, ws=64, wsc=None, dt=capi.BF16, bias=None, res=None,
                  rs=32, od=capi.BF16, T=4, N=32, K=64, act=capi.ACT_NONE, y=2 * FAR, ys=32,
                  z=None, zs=32, err=None, stream=None)
COMMON_FWD = [
    (dict(dt=capi.F32, od=capi.F32), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(od=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(od=capi.E4M3, dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(T=-1), capi.ERR_INVALID_ARG),
    (dict(N=0), capi.ERR_INVALID_ARG),
    (dict(K=0), capi.ERR_INVALID_ARG),
    (dict(K=63), capi.ERR_INVALID_ARG),                  # not whole 16-byte units
    (dict(act=5), capi.ERR_INVALID_ARG),
    (dict(act=-1), capi.ERR_INVALID_ARG),
    (dict(xs=56), capi.ERR_INVALID_ARG),
    (dict(xs=68), capi.ERR_INVALID_ARG),
    (dict(ws=66), capi.ERR_INVALID_ARG),
    (dict(ys=31), capi.ERR_INVALID_ARG),
    (dict(x=None), capi.ERR_INVALID_ARG),
    (dict(w=None), capi.ERR_INVALID_ARG),
    (dict(y=None), capi.ERR_INVALID_ARG),
    (dict(xsc=P), capi.ERR_INVALID_ARG),                 # scales without e4m3
    (dict(dt=capi.E4M3), capi.ERR_INVALID_ARG),          # e4m3 without scales
    (dict(dt=capi.E4M3, xsc=P), capi.ERR_INVALID_ARG),
    (dict(dt=capi.E4M3, xsc=P, wsc=P, K=8), capi.ERR_INVALID_ARG),
    (dict(y=P), capi.ERR_INVALID_ARG),                   # y over x
    (dict(y=FAR + 64), capi.ERR_INVALID_ARG),            # y over the weight
    (dict(z=2 * FAR, zs=64), capi.ERR_INVALID_ARG),      # preact over y
    (dict(x=P + 8), capi.ERR_MISALIGNED),
    (dict(w=FAR + 2), capi.ERR_MISALIGNED),
    (dict(y=2 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(err=P + 2), capi.ERR_MISALIGNED),
    (dict(T=1 << 31), capi.ERR_TOO_LARGE),
    (dict(N=1 << 30, ys=1 << 31, zs=1 << 32), capi.ERR_TOO_LARGE),
    (dict(K=1 << 31, xs=1 << 31, ws=1 << 31), capi.ERR_TOO_LARGE),
    (dict(xs=1 << 40), capi.ERR_TOO_LARGE),
]


@pytest.mark.parametrize("kw,code", COMMON_FWD + [
    (dict(res=3 * FAR, rs=31), capi.ERR_INVALID_ARG),
    (dict(res=2 * FAR, rs=40), capi.ERR_INVALID_ARG),    # in place with another stride
    (dict(z=3 * FAR, res=3 * FAR), capi.ERR_INVALID_ARG),
    (dict(z=3 * FAR, zs=31), capi.ERR_INVALID_ARG),
    (dict(bias=P + 1), capi.ERR_MISALIGNED),
])
def test_linear_fwd_refuses(lib, kw, code):
    assert lib.linear_fwd(*args(LINEAR_FWD, kw)) == code


GLU_FWD = {k: v for k, v in LINEAR_FWD.items() if k not in ("bias", "res", "rs")}
GLU_FWD.update(act=capi.ACT_SILU, zs=64)


@pytest.mark.parametrize("kw,code", COMMON_FWD + [
    (dict(act=capi.ACT_NONE), capi.ERR_INVALID_ARG),
    (dict(z=3 * FAR, zs=63), capi.ERR_INVALID_ARG),
])
def test_glu_fwd_refuses(lib, kw, code):
    assert lib.glu_fwd(*args(GLU_FWD, kw)) == code


LINEAR_BWD = dict(dy=P, dys=32, x=FAR, xs=64, w=2 * FAR, ws=64, z=3 * FAR, zs=32, dt=capi.BF16,
                  T=4, N=32, K=64, act=capi.ACT_SILU, dx=4 * FAR, dxs=64, dw=5 * FAR, dwd=capi.F32,
                  db=P, acc=0, err=None, work=6 * FAR, workb=1 << 20, stream=None)
COMMON_BWD = [
    (dict(dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(dwd=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(T=-1), capi.ERR_INVALID_ARG),
    (dict(K=60), capi.ERR_INVALID_ARG),
    (dict(act=9), capi.ERR_INVALID_ARG),
    (dict(z=None), capi.ERR_INVALID_ARG),
    (dict(zs=31), capi.ERR_INVALID_ARG),
    (dict(dy=None), capi.ERR_INVALID_ARG),
    (dict(x=None), capi.ERR_INVALID_ARG),
    (dict(w=None), capi.ERR_INVALID_ARG),
    (dict(xs=60), capi.ERR_INVALID_ARG),
    (dict(dxs=63), capi.ERR_INVALID_ARG),
    (dict(acc=1, dwd=capi.BF16), capi.ERR_INVALID_ARG),  # accumulation is fp32
    (dict(dx=P), capi.ERR_INVALID_ARG),                  # dx over dy
    (dict(dw=FAR), capi.ERR_INVALID_ARG),                # dweight over x
    (dict(dx=5 * FAR), capi.ERR_INVALID_ARG),            # dx over dweight
    (dict(dx=4 * FAR + 2), capi.ERR_MISALIGNED),
    (dict(dxs=65), capi.ERR_MISALIGNED),
    (dict(dw=5 * FAR + 4), capi.ERR_MISALIGNED),
    (dict(work=None), capi.ERR_WORKSPACE_TOO_SMALL),
    (dict(workb=64), capi.ERR_WORKSPACE_TOO_SMALL),
    (dict(work=6 * FAR + 16), capi.ERR_MISALIGNED),
]


@pytest.mark.parametrize("kw,code", COMMON_BWD + [
    (dict(dx=None, dw=None, db=None), capi.ERR_INVALID_ARG),
    (dict(db=P + 2), capi.ERR_MISALIGNED),
])
def test_linear_bwd_refuses(lib, kw, code):
    assert lib.linear_bwd(*args(LINEAR_BWD, kw)) == code


GLU_BWD = {k: v for k, v in LINEAR_BWD.items() if k != "db"}
GLU_BWD.update(zs=64)


@pytest.mark.parametrize("kw,code", COMMON_BWD + [
    (dict(act=capi.ACT_NONE), capi.ERR_INVALID_ARG),
    (dict(dx=None, dw=None), capi.ERR_INVALID_ARG),
])
def test_glu_bwd_refuses(lib, kw, code):
    assert lib.glu_bwd(*args(GLU_BWD, kw)) == code


def test_workspace_sizes(lib):
    assert lib.vlmce_rmsnorm_bwd_workspace_bytes(0, 64) > 0
    assert lib.vlmce_rmsnorm_bwd_workspace_bytes(-1, 64) == 0
    assert lib.vlmce_rmsnorm_bwd_workspace_bytes(4, 0) == 0
    assert lib.vlmce_linear_bwd_workspace_bytes(100, 30, 64) >= 2 * 100 * 32
    assert lib.vlmce_glu_bwd_workspace_bytes(100, 30, 64) >= 2 * 100 * 64
    assert lib.vlmce_linear_bwd_workspace_bytes(4, 0, 64) == 0
    assert lib.vlmce_glu_bwd_workspace_bytes(4, 8, -8) == 0
