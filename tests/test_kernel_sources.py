"""Properties of the kernels' sources that no call shows reliably.  CPU only."""
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "vocabulary_lm_cross_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", ["gemm.cuh", "mm_pair.cuh", "mm_large.cuh", "mm_grad.cuh", "mm_small.cuh"])
def test_no_warp_waits_only_for_the_lanes_that_happen_to_be_together(name):
    # after a wait loop the lanes of a warp may be apart: a mask of the active ones would
    # let a lane give a slot back that another has yet to read
    assert "__activemask" not in source(name)
