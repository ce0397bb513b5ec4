"""Sizes and overlaps that the experts' entry points refuse on the host, where a kernel's
arithmetic or its order of reads and writes would not hold.  CPU only: no compute call is
made (fake, suitably aligned device addresses; every call below fails its checks)."""
import pytest

from tests.test_layers_capi import args
from tests.test_moe_capi import SORT
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
