"""Products whose K two to eight CTAs share, also where their number divides neither the
tile's rows nor the blocks of K; bounds as in test_block_linear_gpu.py."""
import numpy as np
import pytest
import torch

import vocabulary_lm_cross_gb300 as v
from oracle import moe as om
from tests.layers_parity import DT, f64, gen, randn
from tests.test_block_linear_gpu import blocks, bound, check_dense, e4m3, near, scales

pytestmark = pytest.mark.gpu

# (T, N, K): tiles of 16, 32, 64 and 128 rows
DENSE = [(33, 4932, 2484), (1, 6057, 1536), (1, 6407, 1296), (3, 78, 1084), (1, 591, 668), (5, 591, 668), (1, 128, 896),
         (1, 168, 924), (67, 5159, 2463), (51, 4914, 1040), (33, 4298, 2040), (18, 6485, 1808), (25, 4892, 1948),
         (18, 5162, 1552), (219, 388, 2826), (38, 6484, 2527), (50, 5205, 3204), (35, 4270, 4124), (226, 816, 1808),
         (65, 7889, 5043), (376, 1580, 2178), (165, 2184, 3348), (103, 3393, 2505), (351, 834, 5048)]
# (E, T, N, K)
EXPERTS = [(3, 3, 4443, 5820), (1, 1, 6187, 1296), (5, 4, 1563, 1296), (2, 8, 52, 1180), (1, 1, 69, 668), (3, 1, 161, 828),
           (1, 1, 79, 1948), (5, 77, 2767, 3222), (5, 188, 1284, 1084), (5, 400, 391, 2048), (2, 390, 393, 1555),
           (5, 393, 292, 1948), (2, 297, 391, 1596), (2, 163, 515, 2874), (5, 208, 1500, 2438), (3, 314, 530, 4370),
           (3, 259, 519, 5561), (2, 191, 2948, 4511), (1, 388, 1558, 2530), (2, 297, 1170, 3465)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vocabulary_lm_cross_gb300 import build
    build.build()


@pytest.fixture(autouse=True)
def _no_errors():
    yield
    v.check_device_errors()


def test_every_split_is_reached():
    for plans in ([v.describe_block_linear_plan(T, N, K) for T, N, K in DENSE],
                  [v.describe_block_linear_plan(T, N, K, E) for E, T, N, K in EXPERTS]):
        assert {2, 3, 4, 5, 6, 7, 8} <= {p.split for p in plans}
        assert {16, 32, 64, 128} <= {p.rows for p in plans if p.split > 1}


@pytest.mark.parametrize("by_row", [False, True])
@pytest.mark.parametrize("T,N,K", DENSE)
def test_dense(T, N, K, by_row):
    check_dense(T, N, K, "f16" if T % 2 else "bf16", by_row, residual=N % 2 == 0, pad=K % 3)


@pytest.mark.parametrize("E,T,N,K", EXPERTS)
def test_experts(E, T, N, K):
    g = gen(E + T + N + K)
    cut = torch.randint(0, T + 1, (E - 1,), generator=g).sort().values.tolist()
    off = np.array([0, *cut, T])
    by_row, dtype = T % 2 == 1, "f16" if N % 2 else "bf16"
    x, xs = e4m3(g, T, K), scales(g, T, blocks(K))
    w, ws = e4m3(g, N, K, 0, (E,)), scales(g, N if by_row else blocks(N), blocks(K), 0, (E,))
    res = randn(g, (T, N), DT[dtype], sigma=5.0) if K % 2 else None
    got = v.block_linear_fwd(x, xs, w, ws, res, offsets=torch.from_numpy(off).int().cuda(), out_dtype=DT[dtype])
    want, size = np.zeros((T, N)), np.zeros((T, N))
    for e in range(E):
        r = slice(off[e], off[e + 1])
        want[r], size[r] = om.product(f64(x[r].float()), f64(xs[r]), f64(w[e].float()), f64(ws[e]), 1 if by_row else 128)
    if res is not None:
        want, size = want + f64(res), size + np.abs(f64(res))
    near(got, want, dtype, bound(size, K), "y")
