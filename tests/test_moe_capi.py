"""The experts' entry points, quantize_blocks and the block-scaled products refuse bad
arguments on the host before anything is enqueued.  CPU only: no compute call is made
(fake, suitably aligned device addresses; every call below fails its checks)."""
import pytest

from tests.test_layers_capi import FAR, P, args
from vocabulary_lm_cross_gb300 import build, capi

BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


def test_rows_of_any_choice(lib):
    assert lib.vlmce_moe_rows(0, 2, 8, 128) == 0
    assert lib.vlmce_moe_rows(10, 2, 8, 1) == 20
    assert lib.vlmce_moe_rows(1, 2, 8, 128) == 256       # two experts at most
    assert lib.vlmce_moe_rows(1000, 2, 8, 128) == (2000 + 8 * 127) // 128 * 128
    for bad in ((-1, 2, 8, 1), (1, 0, 8, 1), (1, 2, 0, 1), (1, 2, 8, 0), (1, 65, 8, 1), (1, 2, 1025, 1),
                (1 << 31, 1, 8, 1), (1 << 20, 2, 1024, 1 << 30), (1, 1, 1, 1 << 31)):
        assert lib.vlmce_moe_rows(*bad) == -1, bad


SORT = dict(ids=P, ld=2, wide=1, T=8, k=2, E=4, align=1, pos=FAR, off=2 * FAR, cnt=3 * FAR, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), capi.ERR_INVALID_ARG), (dict(k=0), capi.ERR_INVALID_ARG), (dict(E=0), capi.ERR_INVALID_ARG),
    (dict(align=0), capi.ERR_INVALID_ARG), (dict(ld=1), capi.ERR_INVALID_ARG),
    (dict(ids=None), capi.ERR_INVALID_ARG), (dict(pos=None), capi.ERR_INVALID_ARG),
    (dict(off=None), capi.ERR_INVALID_ARG), (dict(cnt=None), capi.ERR_INVALID_ARG),
    (dict(pos=P), capi.ERR_INVALID_ARG), (dict(off=P), capi.ERR_INVALID_ARG), (dict(cnt=P + 64), capi.ERR_INVALID_ARG),
    (dict(off=FAR + 8), capi.ERR_INVALID_ARG), (dict(cnt=2 * FAR + 16), capi.ERR_INVALID_ARG),
    (dict(ids=P + 4), capi.ERR_MISALIGNED), (dict(wide=0, ids=P + 2), capi.ERR_MISALIGNED),
    (dict(pos=FAR + 2), capi.ERR_MISALIGNED), (dict(off=2 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(k=65, ld=65), capi.ERR_TOO_LARGE), (dict(E=1025), capi.ERR_TOO_LARGE),
    (dict(T=1 << 30), capi.ERR_TOO_LARGE), (dict(align=1 << 31), capi.ERR_TOO_LARGE),
    (dict(align=1 << 30), capi.ERR_TOO_LARGE), (dict(ld=BIG), capi.ERR_TOO_LARGE),
])
def test_moe_sort_refuses(lib, kw, code):
    assert lib.moe_sort(*args(SORT, kw)) == code


GATHER = dict(x=P, xs=64, dt=capi.BF16, pos=6 * FAR, off=7 * FAR, cnt=8 * FAR, T=8, k=2, E=4, R=16, H=64,
              rows=2 * FAR, rs=64, rd=capi.BF16, scale=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE), (dict(rd=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(T=-1), capi.ERR_INVALID_ARG), (dict(R=-1), capi.ERR_INVALID_ARG), (dict(H=0), capi.ERR_INVALID_ARG),
    (dict(k=0), capi.ERR_INVALID_ARG), (dict(E=0), capi.ERR_INVALID_ARG), (dict(xs=63), capi.ERR_INVALID_ARG),
    (dict(rs=63), capi.ERR_INVALID_ARG), (dict(x=None), capi.ERR_INVALID_ARG), (dict(rows=None), capi.ERR_INVALID_ARG),
    (dict(pos=None), capi.ERR_INVALID_ARG), (dict(off=None), capi.ERR_INVALID_ARG), (dict(cnt=None), capi.ERR_INVALID_ARG),
    (dict(rd=capi.E4M3), capi.ERR_INVALID_ARG), (dict(scale=3 * FAR), capi.ERR_INVALID_ARG),
    (dict(rows=P), capi.ERR_INVALID_ARG), (dict(rd=capi.E4M3, scale=2 * FAR + 64), capi.ERR_INVALID_ARG),
    (dict(rd=capi.E4M3, scale=P), capi.ERR_INVALID_ARG), (dict(rows=6 * FAR), capi.ERR_INVALID_ARG),
    (dict(x=P + 1), capi.ERR_MISALIGNED), (dict(rows=2 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(pos=6 * FAR + 2), capi.ERR_MISALIGNED), (dict(rd=capi.E4M3, scale=3 * FAR + 2), capi.ERR_MISALIGNED),
    (dict(R=1 << 31), capi.ERR_TOO_LARGE), (dict(H=1 << 25, xs=1 << 25, rs=1 << 25), capi.ERR_TOO_LARGE),
    (dict(xs=BIG), capi.ERR_TOO_LARGE), (dict(rs=BIG), capi.ERR_TOO_LARGE), (dict(k=65), capi.ERR_TOO_LARGE),
    (dict(E=1025), capi.ERR_TOO_LARGE),
])
def test_moe_gather_refuses(lib, kw, code):
    assert lib.moe_gather(*args(GATHER, kw)) == code


COMBINE = dict(rows=P, rs=64, dt=capi.BF16, pos=6 * FAR, w=FAR, ws=2, wd=capi.F32, res=None, ress=64, T=8, k=2, R=16,
               H=64, y=2 * FAR, ys=64, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE), (dict(wd=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(T=-1), capi.ERR_INVALID_ARG), (dict(rs=63), capi.ERR_INVALID_ARG), (dict(ys=63), capi.ERR_INVALID_ARG),
    (dict(ws=1), capi.ERR_INVALID_ARG), (dict(res=3 * FAR, ress=63), capi.ERR_INVALID_ARG),
    (dict(rows=None), capi.ERR_INVALID_ARG), (dict(y=None), capi.ERR_INVALID_ARG), (dict(pos=None), capi.ERR_INVALID_ARG),
    (dict(y=P), capi.ERR_INVALID_ARG), (dict(y=FAR), capi.ERR_INVALID_ARG), (dict(y=6 * FAR), capi.ERR_INVALID_ARG),
    (dict(res=2 * FAR, ress=72), capi.ERR_INVALID_ARG), (dict(rows=P + 1), capi.ERR_MISALIGNED),
    (dict(w=FAR + 2), capi.ERR_MISALIGNED), (dict(y=2 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(ws=BIG), capi.ERR_TOO_LARGE), (dict(R=1 << 31), capi.ERR_TOO_LARGE),
])
def test_moe_combine_refuses(lib, kw, code):
    assert lib.moe_combine(*args(COMBINE, kw)) == code


COMBINE_BWD = dict(dy=P, ds=64, rows=FAR, rs=64, dt=capi.BF16, pos=6 * FAR, off=7 * FAR, cnt=8 * FAR, w=2 * FAR, ws=2,
                   wd=capi.F32, T=8, k=2, E=4, R=16, H=64, drows=3 * FAR, drs=64, dw=4 * FAR, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE), (dict(wd=capi.F16), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(drows=None, dw=None), capi.ERR_INVALID_ARG), (dict(dy=None), capi.ERR_INVALID_ARG),
    (dict(rows=None), capi.ERR_INVALID_ARG), (dict(ds=63), capi.ERR_INVALID_ARG), (dict(drs=63), capi.ERR_INVALID_ARG),
    (dict(drows=P), capi.ERR_INVALID_ARG), (dict(drows=FAR), capi.ERR_INVALID_ARG),
    (dict(dw=3 * FAR), capi.ERR_INVALID_ARG), (dict(dw=2 * FAR), capi.ERR_INVALID_ARG),
    (dict(dw=6 * FAR), capi.ERR_INVALID_ARG), (dict(off=None), capi.ERR_INVALID_ARG),
    (dict(dw=4 * FAR + 2), capi.ERR_MISALIGNED), (dict(drows=3 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(cnt=8 * FAR + 2), capi.ERR_MISALIGNED), (dict(drs=BIG), capi.ERR_TOO_LARGE),
])
def test_moe_combine_bwd_refuses(lib, kw, code):
    assert lib.moe_combine_bwd(*args(COMBINE_BWD, kw)) == code


QUANT = dict(x=P, dt=capi.BF16, batch=1, R=256, C=256, xs=256, xb=0, square=0, q=FAR, qs=256, s=2 * FAR, qt=3 * FAR,
             qts=256, st=4 * FAR, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE), (dict(batch=-1), capi.ERR_INVALID_ARG),
    (dict(R=-1), capi.ERR_INVALID_ARG), (dict(C=0), capi.ERR_INVALID_ARG), (dict(xs=255), capi.ERR_INVALID_ARG),
    (dict(qs=255), capi.ERR_INVALID_ARG), (dict(qts=255), capi.ERR_INVALID_ARG),
    (dict(s=None), capi.ERR_INVALID_ARG), (dict(q=None), capi.ERR_INVALID_ARG), (dict(st=None), capi.ERR_INVALID_ARG),
    (dict(q=None, s=None, qt=None, st=None), capi.ERR_INVALID_ARG), (dict(x=None), capi.ERR_INVALID_ARG),
    (dict(batch=2, xb=100), capi.ERR_INVALID_ARG), (dict(q=P), capi.ERR_INVALID_ARG),
    (dict(qt=FAR + 256), capi.ERR_INVALID_ARG), (dict(s=4 * FAR), capi.ERR_INVALID_ARG),
    (dict(x=P + 1), capi.ERR_MISALIGNED), (dict(s=2 * FAR + 2), capi.ERR_MISALIGNED),
    (dict(st=4 * FAR + 1), capi.ERR_MISALIGNED), (dict(R=1 << 31, qts=1 << 31), capi.ERR_TOO_LARGE),
    (dict(xs=1 << 50), capi.ERR_TOO_LARGE), (dict(qs=1 << 50), capi.ERR_TOO_LARGE),
    (dict(batch=1 << 31, xb=1 << 20), capi.ERR_TOO_LARGE),
])
def test_quantize_blocks_refuses(lib, kw, code):
    assert lib.quantize_blocks(*args(QUANT, kw)) == code


FWD = dict(x=P, xs=256, xsc=FAR, xss=2, w=2 * FAR, ws=256, wsc=3 * FAR, wss=2, block=128, off=None, E=1, res=None, rs=64,
           od=capi.BF16, T=32, N=64, K=256, y=4 * FAR, ys=64, err=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(od=capi.F32), capi.ERR_UNSUPPORTED_DTYPE), (dict(od=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE),
    (dict(block=64), capi.ERR_INVALID_ARG), (dict(E=2), capi.ERR_INVALID_ARG),  # experts without offsets
    (dict(off=P, E=0), capi.ERR_INVALID_ARG), (dict(T=-1), capi.ERR_INVALID_ARG), (dict(N=0), capi.ERR_INVALID_ARG),
    (dict(K=0), capi.ERR_INVALID_ARG), (dict(xs=240), capi.ERR_INVALID_ARG), (dict(xs=264), capi.ERR_INVALID_ARG),
    (dict(ws=258), capi.ERR_INVALID_ARG), (dict(xss=1), capi.ERR_INVALID_ARG), (dict(wss=1), capi.ERR_INVALID_ARG),
    (dict(ys=63), capi.ERR_INVALID_ARG), (dict(res=5 * FAR, rs=63), capi.ERR_INVALID_ARG),
    (dict(x=None), capi.ERR_INVALID_ARG), (dict(xsc=None), capi.ERR_INVALID_ARG), (dict(w=None), capi.ERR_INVALID_ARG),
    (dict(wsc=None), capi.ERR_INVALID_ARG), (dict(y=None), capi.ERR_INVALID_ARG), (dict(y=P), capi.ERR_INVALID_ARG),
    (dict(y=FAR), capi.ERR_INVALID_ARG), (dict(y=2 * FAR), capi.ERR_INVALID_ARG), (dict(y=3 * FAR), capi.ERR_INVALID_ARG),
    (dict(off=4 * FAR + 64), capi.ERR_INVALID_ARG), (dict(res=4 * FAR, rs=72), capi.ERR_INVALID_ARG),
    (dict(x=P + 8), capi.ERR_MISALIGNED), (dict(w=2 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(xsc=FAR + 2), capi.ERR_MISALIGNED), (dict(y=4 * FAR + 1), capi.ERR_MISALIGNED),
    (dict(off=P + 2), capi.ERR_MISALIGNED), (dict(err=P + 2), capi.ERR_MISALIGNED),
    (dict(off=P, E=1025), capi.ERR_TOO_LARGE), (dict(T=1 << 31), capi.ERR_TOO_LARGE),
    (dict(N=1 << 31, ys=1 << 31), capi.ERR_TOO_LARGE), (dict(off=P, E=1024, N=1 << 21, ys=1 << 21), capi.ERR_TOO_LARGE),
    (dict(xs=1 << 40), capi.ERR_TOO_LARGE), (dict(T=1 << 30, N=1 << 20, ys=1 << 20), capi.ERR_TOO_LARGE),
])
def test_block_linear_fwd_refuses(lib, kw, code):
    assert lib.block_linear_fwd(*args(FWD, kw)) == code


DW = dict(d=P, ds=256, dsc=FAR, dss=2, x=2 * FAR, xs=256, xsc=3 * FAR, xss=2, off=None, E=1, R=256, N=64, K=32, dw=4 * FAR,
          dt=capi.F32, acc=0, err=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=capi.E4M3), capi.ERR_UNSUPPORTED_DTYPE), (dict(E=2), capi.ERR_INVALID_ARG),
    (dict(R=-1), capi.ERR_INVALID_ARG), (dict(N=0), capi.ERR_INVALID_ARG), (dict(K=0), capi.ERR_INVALID_ARG),
    (dict(dt=capi.BF16, acc=1), capi.ERR_INVALID_ARG), (dict(ds=255), capi.ERR_INVALID_ARG),
    (dict(xs=264), capi.ERR_INVALID_ARG), (dict(dss=1), capi.ERR_INVALID_ARG), (dict(xss=1), capi.ERR_INVALID_ARG),
    (dict(d=None), capi.ERR_INVALID_ARG), (dict(x=None), capi.ERR_INVALID_ARG), (dict(dw=None), capi.ERR_INVALID_ARG),
    (dict(dsc=None), capi.ERR_INVALID_ARG), (dict(dw=P), capi.ERR_INVALID_ARG), (dict(dw=FAR), capi.ERR_INVALID_ARG),
    (dict(off=4 * FAR), capi.ERR_INVALID_ARG), (dict(d=P + 8), capi.ERR_MISALIGNED), (dict(dw=4 * FAR + 2), capi.ERR_MISALIGNED),
    (dict(off=P + 1), capi.ERR_MISALIGNED), (dict(R=1 << 31, ds=1 << 31, xs=1 << 31), capi.ERR_TOO_LARGE),
    (dict(off=P, E=1024, N=1 << 20, K=1 << 20), capi.ERR_TOO_LARGE),
    (dict(ds=1 << 40), capi.ERR_TOO_LARGE),
])
def test_block_linear_dweight_refuses(lib, kw, code):
    assert lib.block_linear_dweight(*args(DW, kw)) == code
