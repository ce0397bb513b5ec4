"""Properties of the expert kernels' sources that no call shows reliably.  CPU only."""
import glob
import os
import re

from tests.test_kernel_sources import CSRC, source


def test_arrivals_at_another_ctas_barrier_name_the_clusters_scope():
    # without a scope, an arrival counts within its own CTA only, and orders nothing for a
    # wait in another one
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        for op in re.findall(r"mbarrier\.arrive[a-z0-9_:.]*shared::cluster[a-z0-9_:.]*", source(os.path.basename(path))):
            assert ".cluster.shared::cluster" in op, (path, op)


def test_the_pairs_issuer_waits_at_the_clusters_scope_for_what_both_ctas_give_back():
    waits = re.findall(r"wait_bar(<true>)?\(buf_empty", source("mm_block_pair.cuh"))
    assert waits and all(w == "<true>" for w in waits)
