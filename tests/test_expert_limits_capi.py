"""Sizes and overlaps that the experts' entry points refuse on the host, where a kernel's
arithmetic or its order of reads and writes would not hold.  CPU only: no compute call is
made (fake, suitably aligned device addresses; every call below fails its checks)."""
import pytest

from tests.test_layers_capi import args
from tests.test_moe_capi import COMBINE_BWD, FAR, GATHER, SORT
from vocabulary_lm_cross_gb300 import build, capi

PAIRS = 2 ** 31 - 512  # whose numbers, a warp's 512 further on included, fit in 32 bits


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.lib()


@pytest.mark.parametrize("T,k,E", [(PAIRS + 1, 1, 1), (2 ** 31 - 2, 1, 1), (PAIRS // 8 + 1, 8, 256), (268435400, 8, 256),
                                   (PAIRS // 64 + 1, 64, 100)])
def test_sort_ends_where_its_numbers_of_pairs_do(lib, T, k, E):
    assert T * k + E <= 2 ** 31 - 1  # the rows themselves would fit
    assert lib.vlmce_moe_rows(T, k, E, 1) == -1
    assert lib.moe_sort(*args(SORT, dict(T=T, k=k, E=E, ld=k, pos=1 << 40, off=1 << 50, cnt=1 << 51))) == capi.ERR_TOO_LARGE


@pytest.mark.parametrize("T,k,E", [(PAIRS, 1, 1), (PAIRS, 1, 510), (PAIRS // 8, 8, 256), (PAIRS // 64, 64, 100)])
def test_rows_of_the_largest_sorts(lib, T, k, E):
    assert lib.vlmce_moe_rows(T, k, E, 1) == T * k


# (GATHER and COMBINE_BWD have five offsets from 7 FAR and four counts from 8 FAR)
@pytest.mark.parametrize("kw", [
    dict(rows=7 * FAR), dict(rows=8 * FAR), dict(rows=7 * FAR + 18), dict(rows=8 * FAR + 14),
    dict(rd=capi.E4M3, scale=7 * FAR), dict(rd=capi.E4M3, scale=8 * FAR + 12),
    dict(rd=capi.E4M3, scale=3 * FAR, rows=8 * FAR), dict(off=2 * FAR + 15 * 128 + 124),
])
def test_gather_writes_no_offsets_and_counts(lib, kw):
    assert lib.moe_gather(*args(GATHER, kw)) == capi.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(drows=7 * FAR), dict(drows=8 * FAR), dict(dw=7 * FAR + 16), dict(dw=8 * FAR + 12), dict(dw=8 * FAR - 60),
    dict(cnt=3 * FAR + 64),
])
def test_combine_bwd_writes_no_offsets_and_counts(lib, kw):
    assert lib.moe_combine_bwd(*args(COMBINE_BWD, kw)) == capi.ERR_INVALID_ARG
