"""The largest order of tokens that moe_sort takes: 2^31 - 512 pairs."""
import pytest
import torch

import vocabulary_lm_cross_gb300 as v

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from vocabulary_lm_cross_gb300 import build
    build.build()


@pytest.mark.parametrize("k", [1, 8])
def test_sort_of_the_most_pairs(k):
    n, E, step = 2 ** 31 - 512, 3, 2 ** 27
    experts = torch.empty(n, dtype=torch.int32, device="cuda")
    for a in range(0, n, step):
        i = torch.arange(a, min(n, a + step), device="cuda")
        experts[a:a + step] = i % E
    order = v.moe_sort(experts.view(n // k, k), E)
    counts = [(n - e + E - 1) // E for e in range(E)]
    offsets = [sum(counts[:e]) for e in range(E + 1)]
    assert order.counts.tolist() == counts and order.offsets.tolist() == offsets and order.rows == n
    start = torch.tensor(offsets[:E], device="cuda")
    flat = order.position.view(-1)
    for a in range(0, n, step):
        i = torch.arange(a, min(n, a + step), device="cuda")
        assert torch.equal(flat[a:a + step].long(), start[i % E] + i // E)
