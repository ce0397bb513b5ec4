"""Properties of the kernels' sources that no call shows reliably.  CPU only."""
import math
import os
import re

import numpy as np
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


def test_the_gelu_fit_is_as_near_as_its_comment_says():
    text = source("act.cuh")
    bound = float(re.search(r"largest\s*(?://)?\s*relative error \(([0-9.e-]+)", text)[1])
    body = text[text.index("float cdf("):text.index("const float q = 0.5f")]
    coef = [np.float32(c) for c in re.findall(r"(?:p = |p, t, )(-?[0-9.]+)f", body)]
    assert len(coef) == 9
    x = np.linspace(0.0, 13.4, 20001)
    t = 1.0 / (1.0 + 0.3 / math.sqrt(2.0) * x)
    p = np.zeros_like(t)
    for c in coef:
        p = p * t + float(c)
    want = np.array([math.exp(a * a / 2) * math.erfc(a / math.sqrt(2.0)) for a in x])
    # (the library functions behind `want` are good to a few 1e-15, times x^2 / 2 = 90)
    assert np.abs(t * p / want - 1).max() <= bound + 1e-12
